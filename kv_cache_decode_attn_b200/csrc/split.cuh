// Pieces shared by the split-KV decode kernels (decode.cu, decode_fp8.cu,
// decode_rows8.cu): the
// launch parameters, the length check, the selection of keys, and the TMA producer
// loop that streams a work item's 64-token K/V tiles into a shared-memory ring.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace kvattn {

// SEL instances, one chunk per sequence (on): the split kernel writes the outputs itself.
struct DirectOut {
  int on = 0, o_bf16 = 0, T = 0, Hq = 0, G = 0;
  void* o = nullptr;      // [B, T, Hq, D]
  float* lse = nullptr;   // [B, Hq, T], or none

  // columns col .. col + 3 of row r = t * G + head of the group, of sequence b and KV head g
  template <int D>
  __device__ __forceinline__ void store4(int b, int g, int r, int col, float4 v) const {
    const int t = r / G, h = g * G + r - t * G;
    const size_t at = (((size_t)b * T + t) * Hq + h) * D + col;
    if (o_bf16) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o) + at) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(o) + at) = v;
    }
  }
  __device__ __forceinline__ void store_lse(int b, int g, int r, float v) const {
    const int t = r / G, h = g * G + r - t * G;
    if (lse) lse[((size_t)b * Hq + h) * T + t] = v;
  }
  // rows r0 .. r1 - 1 as NaN, by threads `thread` of `threads`
  template <int D>
  __device__ __forceinline__ void store_nan(int b, int g, int r0, int r1, int thread, int threads) const {
    for (int i = thread; i < (r1 - r0) * (D / 4); i += threads) {
      const int r = r0 + i / (D / 4), col = i % (D / 4) * 4;
      store4<D>(b, g, r, col, make_float4(NAN, NAN, NAN, NAN));
      if (col == 0) store_lse(b, g, r, NAN);
    }
  }
};

inline DirectOut direct_out(const DecodeLaunch& a) {
  DirectOut d;
  d.on = 1;
  d.o_bf16 = a.o_bf16;
  d.T = a.T;
  d.Hq = a.Hq;
  d.G = a.Hq / a.Hkv;
  d.o = a.o;
  d.lse = a.lse;
  return d;
}

// Log-sum-exp of a row from its reference maximum m (base 2, scale folded in) and the sum l
// of 2^(score - m): -inf where every key weighs nothing, NaN where a score is NaN.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

struct SplitParams {
  const __nv_bfloat16* q;
  const float* k_scale;   // FP8 caches: per-KV-head scales (else unused)
  const float* v_scale;
  const int32_t* seqlens;
  const int32_t* page_table;
  float* part_o;
  float* part_lse;
  unsigned* status;
  int T, Hq, Hkv, G, R;
  int chunk, max_chunks, capacity, max_blocks, num_blocks, max_seqlen;
  float scale_log2;
  int causal;
  int balanced = 0;            // tensor-core balanced split: partials indexed by the plan
  const int* plan = nullptr;   // [B, 3]: first chunk, chunks, chunk length per sequence
  KeySelect sel;               // SEL instances: which keys of a sequence the launch reads
  DirectOut out;
  int B = 0;
  int stream = 0;              // SEL instances, > 0: CTAs per KV head that share its tiles evenly (see StreamPlan)
  int early = 0;               // SEL instances: let the next kernel start at once; it waits for this one
  int fence = 0;               // SEL instances: one CTA more, which only waits for the kernel before
};

__device__ __forceinline__ bool seqlen_bad(int L, int T, int max_seqlen, bool paged, int capacity, int max_blocks) {
  if (L < T || L > max_seqlen) return true;
  if (!paged && L > capacity) return true;
  if (paged && (L + kPageTokens - 1) / kPageTokens > max_blocks) return true;
  return false;
}

// The keys sequence b attends to in this launch.  Plain instances (SEL false): its
// first L.  SEL instances number the selected keys consecutively, at the granularity
// of 16-token blocks: number v is position v below s16 (the first tokens that stay
// visible, rounded up to whole blocks) and position v + gap from there on, where gap,
// a multiple of 16, skips the blocks that no query of the call sees.  Chunks, tiles
// and masks all work on these numbers; only the copies map them to positions.
// bad: the sequence's length is invalid for the call.
struct SeqKeys {
  int L;     // selected keys (the last block's tail excluded)
  int s16;   // numbers below it are positions
  int gap;   // position - number from s16 on
  bool bad;
};

// Physical block of a sequence's logical block `blk` (SEL instances).  PREFIX: the first
// sel.prefix_blocks are the shared prefix's.  The producers have a loop each for the two: asked block
// by block, the question alone cost 8 sequences behind a window of 450 (FP8) 1 us of 10.7.
template <bool PREFIX>
__device__ __forceinline__ int block_id(const KeySelect& sel, const int32_t* table_row, int blk) {
  return __ldg(PREFIX && blk < sel.prefix_blocks ? sel.prefix + blk : table_row + blk);
}

template <bool SEL>
__device__ __forceinline__ SeqKeys seq_keys(const KeySelect& sel, const int32_t* seqlens, int b, int T, int max_seqlen,
                                            bool paged, int capacity, int max_blocks) {
  SeqKeys k;
  k.s16 = 0;
  k.gap = 0;
  if constexpr (!SEL) {
    k.L = seqlens[b];
    k.bad = seqlen_bad(k.L, T, max_seqlen, paged, capacity, max_blocks);
  } else {
    if (sel.fixed_len) {           // every sequence's queries against the shared prefix
      k.L = sel.fixed_len;
      k.bad = false;
      return k;
    }
    k.L = seqlens[b];
    k.bad = seqlen_bad(k.L, T, max_seqlen, paged, capacity, max_blocks) || k.L < sel.min_len;
    if (k.bad) return k;
    if (sel.skip) {
      k.gap = sel.skip;
    } else {
      k.s16 = (sel.sinks + kPageTokens - 1) & ~(kPageTokens - 1);
      // first block of the first query's window
      const int w0 = max(0, k.L - T - sel.window + 1) & ~(kPageTokens - 1);
      k.gap = max(0, w0 - k.s16);
    }
    k.L -= k.gap;
  }
  return k;
}

// Even shares (SEL instances, p.stream CTAs per KV head).  For each KV head the launch's
// 64-token tiles stand in one line, sequence after sequence, and CTA i of the head's n
// takes total / n consecutive tiles, the first total % n CTAs one more: even shares
// whatever the lengths, and the ring runs on across the sequences of a share.  With a fixed
// chunk length the items came to 2.2 waves of CTAs for a window of 1024 (16 x 8 pairs), and
// two in five slots idled.  Block c is CTA c / Hkv of head c % Hkv: the heads of a token,
// which lie side by side in the cache, are read at about the same time.  Piece (CTA i of
// head g, sequence b) has partial number g * (n + B) + i + b: along a line each step raises
// i or b, so the numbers are distinct, and those of one sequence are consecutive.
constexpr int kStreamMaxB = 128;   // sequences whose tile counts are summed in shared memory
struct StreamPlan {
  int first[kStreamMaxB + 1];   // tiles (per KV head) of the sequences before
  int len[kStreamMaxB];         // keys of the sequences (seqlens)
};

// First tile of CTA i's share, and the CTA that tile x belongs to.
__device__ __forceinline__ int stream_begin(int i, int n, int total) {
  return i * (total / n) + min(i, total % n);
}
__device__ __forceinline__ int stream_cta(int x, int n, int total) {
  const int share = total / n, wide = total % n * (share + 1);   // tiles of the CTAs with one more
  return x < wide ? x / (share + 1) : (x - total % n) / share;
}

// One warp (the producer): tile counts of the sequences, summed (0 for an invalid length,
// which block 0 reports).  The CTA's other warps wait for it in stream_plan_wait, while
// this one goes on to its first copies.
template <bool PAGED, int kThreads>
__device__ __forceinline__ void stream_plan(const SplitParams& p, StreamPlan* plan) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) plan->first[0] = 0;
  int carry = 0;
  for (int base = 0; base < p.B; base += 32) {
    const int i = base + lane;
    int v = 0;
    if (i < p.B) {
      if (!p.sel.fixed_len) plan->len[i] = p.seqlens[i];
      const SeqKeys k = seq_keys<true>(p.sel, plan->len, i, p.T, p.max_seqlen, PAGED, p.capacity, p.max_blocks);
      if (k.bad && blockIdx.x == 0) atomicOr(p.status, DEV_SEQLEN);
      v = k.bad ? 0 : (k.L + kDecodeTile - 1) / kDecodeTile;
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += u;
    }
    v += carry;
    if (i < p.B) plan->first[i + 1] = v;
    carry = __shfl_sync(0xffffffffu, v, 31);
  }
  __syncwarp();
  asm volatile("barrier.cta.arrive 2, %0;" ::"n"(kThreads) : "memory");
}

template <int kThreads>
__device__ __forceinline__ void stream_plan_wait() {
  asm volatile("barrier.cta.sync 2, %0;" ::"n"(kThreads) : "memory");
}

// A run of consecutive tiles of one (sequence, KV head): keys [tok_begin, tok_end), whose
// partial is number `item`.
struct Segment {
  int b, g, tok_begin, tok_end, n_tiles;
  size_t item;
  SeqKeys sk;
};

// The segment that starts at tile x of the CTA's line, within its share [x, x1).
template <bool PAGED>
__device__ __forceinline__ Segment stream_segment(const SplitParams& p, const StreamPlan* plan, int x, int x1) {
  int lo = 0, hi = p.B - 1;   // the last sequence whose first tile is at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (plan->first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  Segment s;
  s.b = lo;
  s.g = blockIdx.x % p.Hkv;
  const int t0 = x - plan->first[lo];
  s.n_tiles = min(plan->first[lo + 1] - x, x1 - x);
  s.sk = seq_keys<true>(p.sel, plan->len, s.b, p.T, p.max_seqlen, PAGED, p.capacity, p.max_blocks);
  s.tok_begin = t0 * kDecodeTile;
  s.tok_end = min(s.tok_begin + s.n_tiles * kDecodeTile, s.sk.L);
  s.item = (size_t)s.g * (p.stream + p.B) + blockIdx.x / p.Hkv + s.b;
  return s;
}

// One thread: tiles 0 .. n_tiles-1 of keys [tok_begin, tok_end) into the ring of
// C::kStages stages (K then V, C::kHalves 128-byte swizzle spans per token row;
// contiguous: one 64-row box per span; paged: one 16-row box per physical
// block, its page-table entry bounds-checked first; SEL instances: one 16-row box per
// selected block in either layout, both spans of a row in one copy: the stage then holds
// block after block, and each span's 16 rows together), evict-first L2 policy.  A
// stage is refilled once the consumers released it (empty barrier); a wait that
// gives up sets DEV_TIMEOUT and the abort flag.
template <class C, bool PAGED, bool SEL, bool PREFIX = false>
__device__ __forceinline__ void produce_split_tiles(uint8_t* smem, uint64_t* full, uint64_t* empty,
                                                    const CUtensorMap* tmK, const CUtensorMap* tmV,
                                                    const SplitParams& p, int b, int g, int tok_begin, int tok_end,
                                                    int n_tiles, const SeqKeys& sk, int* abort_flag) {
  prefetch_tmap(tmK);
  prefetch_tmap(tmV);
  const uint64_t pol = policy_evict_first();
  for (int i = 0; i < n_tiles; ++i) {
    const int s = i % C::kStages;
    if (i >= C::kStages && !mbar_wait(&empty[s], ((i / C::kStages) - 1) & 1)) {
      atomicOr(p.status, DEV_TIMEOUT);
      *reinterpret_cast<volatile int*>(abort_flag) = 1;
      break;
    }
    uint8_t* kst = smem + s * C::kStageBytes;
    uint8_t* vst = kst + C::kTensorBytes;
    const int t0 = tok_begin + i * kDecodeTile;
    if (!PAGED && !SEL) {
      mbar_arrive_expect_tx(&full[s], C::kStageBytes);
      const int row = b * p.capacity + t0;
#pragma unroll
      for (int h = 0; h < C::kHalves; ++h) {
        tma_load_3d(kst + h * C::kHalfBytes, tmK, &full[s], h * 64, g, row, pol);
        tma_load_3d(vst + h * C::kHalfBytes, tmV, &full[s], h * 64, g, row, pol);
      }
    } else {
      constexpr int kBlocks = kDecodeTile / kPageTokens;
      const int nb = min(kBlocks, (tok_end - t0 + kPageTokens - 1) / kPageTokens);
      const int32_t* row_tab = p.page_table + (size_t)b * p.max_blocks + (SEL ? 0 : t0 / kPageTokens);
      // read the stage's block ids together: the copies' memory clobbers would
      // otherwise serialise one table read per block
      int ids[kBlocks];
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        if constexpr (SEL) {
          const int vt = t0 + j * kPageTokens;
          const int pos = vt + (vt >= sk.s16 ? sk.gap : 0);
          // paged: the block's id; contiguous: its first row in the [B * capacity] view
          ids[j] = j < nb ? (PAGED ? block_id<PREFIX>(p.sel, row_tab, pos / kPageTokens) : b * p.capacity + pos) : 0;
        } else {
          ids[j] = j < nb ? __ldg(row_tab + j) : 0;
        }
      }
      mbar_arrive_expect_tx(&full[s], nb * 2 * C::kHalves * kPageTokens * 128);
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        if (j >= nb) break;
        int blk = ids[j];
        if (PAGED && (blk < 0 || blk >= p.num_blocks)) {
          atomicOr(p.status, DEV_PAGE_ID);
          blk = 0;   // keep the byte count; the result is flagged invalid
        }
        const int row = PAGED ? blk * kPageTokens : blk;
        if constexpr (SEL) {
          tma_load_4d(kst + j * C::kHalves * kPageTokens * 128, tmK, &full[s], 0, g, row, 0, pol);
          tma_load_4d(vst + j * C::kHalves * kPageTokens * 128, tmV, &full[s], 0, g, row, 0, pol);
        } else {
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) {
            tma_load_3d(kst + h * C::kHalfBytes + j * kPageTokens * 128, tmK, &full[s], h * 64, g, row, pol);
            tma_load_3d(vst + h * C::kHalfBytes + j * kPageTokens * 128, tmV, &full[s], h * 64, g, row, pol);
          }
        }
      }
    }
  }
}

// One warp: the tiles of a share [x, x1) of the line, segment after segment, s the first.  Lane j holds
// the first cache row of the segment's block 32 k + j, read while the 32 blocks before are
// being copied: with one thread reading a tile's table entries and then issuing its copies,
// each FP8 tile cost the producer a memory round trip, and the three CTAs of an SM drew
// 4.8 TB/s.  Lane 0 issues the copies (from lanes of their own
// they took 95 cycles each: their operands are warp-uniform, so lanes take turns).
template <class C, bool PAGED, bool PREFIX>
__device__ __forceinline__ void produce_stream(uint8_t* smem, uint64_t* full, uint64_t* empty, const CUtensorMap* tmK,
                                               const CUtensorMap* tmV, const SplitParams& p, const StreamPlan* plan,
                                               Segment s, int x, int x1, int* abort_flag) {
  constexpr int kBlocks = kDecodeTile / kPageTokens;
  const int lane = threadIdx.x & 31;
  const uint64_t pol = policy_evict_first();
  // first row, in the [rows, Hkv, d] view of the cache, of this lane's block of batch k
  auto read_rows = [&](const Segment& s, int k) -> int {
    const int vt = s.tok_begin + (32 * k + lane) * kPageTokens;
    if (vt >= s.tok_end) return 0;
    const int pos = vt + (vt >= s.sk.s16 ? s.sk.gap : 0);
    return PAGED ? block_id<PREFIX>(p.sel, p.page_table + (size_t)s.b * p.max_blocks, pos / kPageTokens)
                 : s.b * p.capacity + pos;
  };
  Segment after = s;
  int next_rows = read_rows(s, 0);
  for (int at = 0;;) {
    x += s.n_tiles;
    int rows = 0;
    for (int i = 0; i < s.n_tiles; ++i, ++at) {
      const int j = i * kBlocks & 31;   // the tile's first block in its batch of 32
      if (j == 0) {
        rows = next_rows;
        if constexpr (PAGED) {
          const bool used = s.tok_begin + (i * kBlocks + lane) * kPageTokens < s.tok_end;
          if (used && (rows < 0 || rows >= p.num_blocks)) {
            atomicOr(p.status, DEV_PAGE_ID);
            rows = 0;   // keep the byte count; the result is flagged invalid
          }
          rows *= kPageTokens;
        }
      }
      int row[kBlocks];
#pragma unroll
      for (int e = 0; e < kBlocks; ++e) row[e] = __shfl_sync(0xffffffffu, rows, j + e);
      const int nb = min(kBlocks, (s.tok_end - (s.tok_begin + i * kDecodeTile) + kPageTokens - 1) / kPageTokens);
      const int st = at % C::kStages;
      bool ok = true;
      if (lane == 0) {
        ok = at < C::kStages || mbar_wait(&empty[st], ((at / C::kStages) - 1) & 1);
        if (ok) {
          mbar_arrive_expect_tx(&full[st], nb * 2 * C::kHalves * kPageTokens * 128);
        } else {
          atomicOr(p.status, DEV_TIMEOUT);
          *reinterpret_cast<volatile int*>(abort_flag) = 1;
        }
      }
      if (!__shfl_sync(0xffffffffu, (int)ok, 0)) return;
      if (lane == 0) {
#pragma unroll
        for (int e = 0; e < kBlocks; ++e) {
          if (e >= nb) break;
          uint8_t* kst = smem + st * C::kStageBytes + e * C::kHalves * kPageTokens * 128;
          tma_load_4d(kst, tmK, &full[st], 0, s.g, row[e], 0, pol);
          tma_load_4d(kst + C::kTensorBytes, tmV, &full[st], 0, s.g, row[e], 0, pol);
        }
      }
      if (j == 0) {   // the batch after this one
        const int k = i * kBlocks / 32 + 1;
        if (k * (32 / kBlocks) < s.n_tiles) {
          next_rows = read_rows(s, k);
        } else if (x < x1) {
          after = stream_segment<PAGED>(p, plan, x, x1);
          next_rows = read_rows(after, 0);
        }
      }
    }
    if (x >= x1) return;
    s = after;
  }
}

// Whether any consumer thread of the CTA (all kThreads of them call this) sees the abort
// flag: one answer for all, so that none waits at a later barrier for one that left.
template <int kThreads>
__device__ __forceinline__ bool consumers_abort(const volatile int* abort_flag) {
  int r;
  asm volatile(
      "{\n"
      ".reg .pred q, r;\n"
      "setp.ne.s32 q, %1, 0;\n"
      "barrier.cta.red.or.pred r, 1, %2, q;\n"
      "selp.s32 %0, 1, 0, r;\n"
      "}\n"
      : "=r"(r)
      : "r"(*abort_flag), "n"(kThreads)
      : "memory");
  return r != 0;
}

// Launch a SEL instance of a warp-level kernel, with one CTA more if p.fence.
template <class Kernel>
inline cudaError_t launch_sel(Kernel kern, int threads, int smem, const CUtensorMap& tk, const CUtensorMap& tv,
                              const SplitParams& sp, int B, cudaStream_t stream) {
  const dim3 grid = sp.stream ? dim3(sp.stream * sp.Hkv + sp.fence) : dim3(sp.max_chunks + sp.fence, sp.Hkv, B);
  return launch_beside(kern, grid, threads, smem, stream, tk, tv, sp);
}

// FP8 caches, at most 8 query rows per KV head: the transposed-product split kernel (decode_fp8.cu)
cudaError_t launch_decode_fp8_rows8(const CUtensorMap& tk, const CUtensorMap& tv, const SplitParams& sp, int B,
                                    bool paged, cudaStream_t stream);
// windowed and shared-prefix decode, at most 8 query rows per KV head (decode_rows8.cu)
cudaError_t launch_decode_rows8(const CUtensorMap& tk, const CUtensorMap& tv, const SplitParams& sp, int B, int d,
                                bool fp8, bool paged, cudaStream_t stream);

}  // namespace kvattn
