// Split-KV decode attention for sm_100a (memory-bound path).
//
// One CTA owns one work item (sequence b, KV head g, key chunk c).  All
// R = (Hq/Hkv) * T query rows that read KV head g are handled together, so each
// K/V byte is streamed from HBM once per step.  A producer warp moves 64-token
// K/V tiles into a shared-memory ring with TMA (128-byte swizzle, evict-first
// L2 policy); consumer warps compute S = Q K^T and O += P V with warp-level bf16
// tensor-core MMAs (fp32 accumulation), keeping a running maximum and running
// denominator per row and rescaling O when the maximum grows.  Each consumer
// warp owns 16 tokens of every tile, so the four warps of a row group are four
// independent online softmaxes that are merged at the end of the chunk.  The
// chunk's normalised output and log-sum-exp go to the workspace; a second
// kernel merges the chunks of each row with the log-sum-exp combine.
//
// FP8 caches (e4m3 codes with one float32 scale per KV head for K and for V):
// the tile is half as many bytes; each consumer thread reads its K and V bytes
// with 16-byte shared loads and converts them exactly to f16 with the hardware
// e4m3x2 -> f16x2 conversion, so the MMAs run in f16 (Q and P are rounded to
// f16).  The sum over d in Q K^T may take the d positions in any order as long
// as Q uses the same order, so a thread's four consecutive K bytes of a row
// feed one k16 step directly; for P V the output columns are permuted the same
// way (column n of the j-th 8-column block is d = 16 n + j) so that a thread's
// V bytes of two keys pair up with one byte permute.  The K scale is folded
// into the softmax scale and the V scale into the chunk's normalisation.
//
// Method: "[BEE-30062] FlashAttention 與高效注意力核心", sections "背景" and
// "為長上下文推論啟用 FlashDecoding" (split along the KV length, numerically
// stable reduction of partial softmax results); "大模型面試笔记——Attention篇"
// section 2 (online safe softmax); "Effizienz", "Der wichtige Maskenfehler beim
// Cache" (bottom-right aligned mask for several new tokens); "KV cache, flash
// attention and inference optimisation" lesson, section "用它" (an FP8 KV cache).
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "split.cuh"

namespace kvattn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int D, int MT, bool FP8>
struct DecodeCfg {
  static_assert(!FP8 || D == 128, "FP8 caches are built for d = 128");
  static_assert(MT == 1 || FP8, "bf16 caches with more than 16 rows run on the tensor-core kernel");
  static constexpr int kConsumerWarps = 4 * MT;
  static constexpr int kThreads = 32 * (kConsumerWarps + 1);
  static constexpr int kHalves = (FP8 ? D : 2 * D) / 128;   // 128-byte swizzle spans per token row
  static constexpr int kHalfBytes = kDecodeTile * 128;
  static constexpr int kTensorBytes = kHalves * kHalfBytes;   // one of K or V per stage
  static constexpr int kStageBytes = 2 * kTensorBytes;
  static constexpr int kBf16Stages = (MT == 1) ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int kStages = FP8 ? 2 * kBf16Stages : kBf16Stages;   // the same bytes in flight
  static constexpr int kRedStride = D + 8;            // floats per row of the merge buffer
  static constexpr int kRedBytes = MT * 4 * 16 * kRedStride * 4;
  static_assert(kRedBytes <= kStages * kStageBytes, "merge buffer must fit in the ring");
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kStatsOffset = kBarOffset + 2 * kStages * 8;
  static constexpr int kSmemBytes = kStatsOffset + MT * 4 * 16 * 2 * 4 + 16 + 1024;  // + alignment slack
  static constexpr int kMinBlocks = (kSmemBytes * 2 <= 227 * 1024) ? 2 : 1;
  // SEL instances merge the warps of a segment while the ring goes on filling: a buffer of
  // its own, for four rows of each row group at a time
  static constexpr int kPassRows = 4;
  static constexpr int kMergeStride = D + 8;
  static constexpr int kMergeOffset = (kSmemBytes - 1024 + 15) / 16 * 16;
  static constexpr int kSelSmemBytes = kMergeOffset + MT * 4 * kPassRows * kMergeStride * 4 + 1024;
  static_assert(kMinBlocks == 1 || 2 * (kSelSmemBytes + (int)sizeof(StreamPlan) + 1024) <= 228 * 1024,
                "two CTAs per SM");
};

// bf16 pair (low = lower index) -> f16 pair
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v) {
  return pack_f16x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <int D, int MT, bool PAGED, bool FP8, bool SEL>
__global__ void __launch_bounds__(DecodeCfg<D, MT, FP8>::kThreads, DecodeCfg<D, MT, FP8>::kMinBlocks)
    decode_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const SplitParams p) {
  using C = DecodeCfg<D, MT, FP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + C::kStages;
  float* stats = reinterpret_cast<float*>(smem + C::kStatsOffset);   // [MT][4][16][2]: m, l
  int* abort_flag = reinterpret_cast<int*>(stats + MT * 4 * 16 * 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  int g = blockIdx.y, b = blockIdx.z;
  int tok_begin, tok_end, n_tiles;
  size_t item;
  SeqKeys sk;
  const StreamPlan* plan = nullptr;
  int x = 0, x1 = 0;   // p.stream: this CTA's share of the tiles
  if constexpr (SEL) {
    if (!p.fence) grid_dependency_wait();   // launched early too; with p.fence the kernel before has waited
    if (p.early) launch_dependents();
    if (p.fence && c == (p.stream ? p.stream * p.Hkv : p.max_chunks)) {
      if (g == 0 && b == 0) grid_dependency_wait();
      return;
    }
  }
  auto init_ring = [&](int thread) {
    if (threadIdx.x == thread) {
      for (int s = 0; s < C::kStages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], C::kConsumerWarps);
      }
      *abort_flag = 0;
      fence_mbar_init();
    }
  };
  if (SEL && p.stream) {
    __shared__ StreamPlan plan_smem;
    init_ring(C::kConsumerWarps * 32);
    if (warp == C::kConsumerWarps) stream_plan<PAGED, C::kThreads>(p, &plan_smem);
    else stream_plan_wait<C::kThreads>();
    plan = &plan_smem;
    const int total = plan->first[p.B], n = min(p.stream, total), i = c / p.Hkv;
    if (i >= n) return;
    x = stream_begin(i, n, total);
    x1 = stream_begin(i + 1, n, total);
  } else {
    sk = seq_keys<SEL>(p.sel, p.seqlens, b, p.T, p.max_seqlen, PAGED, p.capacity, p.max_blocks);
    if (sk.bad) {
      if (threadIdx.x == 0 && c == 0 && g == 0) atomicOr(p.status, DEV_SEQLEN);
      if (SEL && p.out.on) p.out.store_nan<D>(b, g, 0, p.R, threadIdx.x, blockDim.x);
      return;   // else the combine kernel writes NaN rows for this sequence
    }
    tok_begin = c * p.chunk;
    if (tok_begin >= sk.L) return;
    tok_end = min(tok_begin + p.chunk, sk.L);
    n_tiles = (tok_end - tok_begin + kDecodeTile - 1) / kDecodeTile;
    item = ((size_t)b * p.Hkv + g) * p.max_chunks + c;
  }
  float scale_log2 = p.scale_log2, v_scale = 1.f;
  auto bad_scale = [&](int head) {
    if constexpr (!FP8) return false;
    const float ks = __ldg(p.k_scale + head), vs = __ldg(p.v_scale + head);
    return !(ks > 0.f && ks <= 3.402823466e38f && vs > 0.f && vs <= 3.402823466e38f);
  };
  if constexpr (FP8) {
    if (!(SEL && p.stream) && bad_scale(g)) {
      if (threadIdx.x == 0 && c == 0) atomicOr(p.status, DEV_SCALE);
      if (SEL && p.out.on) {
        p.out.store_nan<D>(b, g, 0, p.R, threadIdx.x, blockDim.x);
        return;
      }
      for (int r = threadIdx.x; r < p.R; r += blockDim.x) p.part_lse[item * p.R + r] = NAN;
      return;   // the whole CTA leaves before any barrier: the scales are uniform across it
    }
  }

  if (!(SEL && p.stream)) {   // else the producer has done it, before the plan's barrier
    init_ring(0);
    __syncthreads();
  }

  if (warp == C::kConsumerWarps) {
    // ------------------------------------------------------------ producer
    auto produce = [&](auto prefix) {
      constexpr bool PREFIX = decltype(prefix)::value;
      if (SEL && p.stream) {
        produce_stream<C, PAGED, PREFIX>(smem, full, empty, &tmK, &tmV, p, plan,
                                         stream_segment<PAGED>(p, plan, x, x1), x, x1, abort_flag);
      } else if (lane == 0) {
        produce_split_tiles<C, PAGED, SEL, PREFIX>(smem, full, empty, &tmK, &tmV, p, b, g, tok_begin, tok_end, n_tiles,
                                                   sk, abort_flag);
      }
    };
    if (SEL && PAGED && p.sel.prefix_blocks) produce(std::bool_constant<SEL && PAGED>{});
    else produce(std::false_type{});
    return;
  }

  // -------------------------------------------------------------- consumers
  const int wsub = warp & 3;          // which 16 tokens of each tile
  const int mt = warp >> 2;           // which 16 query rows
  const int gid = lane >> 2, tig = lane & 3;

  // Q fragments of a segment (A operand, 16 x D, row-major) straight from global memory.
  uint32_t qa[D / 16][4];
  auto load_q = [&](int b, int g) {
    const int r0 = mt * 16 + gid, r1 = r0 + 8;
    auto qrow = [&](int r) -> const __nv_bfloat16* {
      const int t = r / p.G, hh = r - t * p.G;
      return p.q + (((size_t)b * p.T + t) * p.Hq + (size_t)g * p.G + hh) * D;
    };
    const __nv_bfloat16* qr0 = r0 < p.R ? qrow(r0) : nullptr;
    const __nv_bfloat16* qr1 = r1 < p.R ? qrow(r1) : nullptr;
    if constexpr (!FP8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int c0 = kk * 16 + tig * 2;
        qa[kk][0] = qr0 ? *reinterpret_cast<const uint32_t*>(qr0 + c0) : 0u;
        qa[kk][1] = qr1 ? *reinterpret_cast<const uint32_t*>(qr1 + c0) : 0u;
        qa[kk][2] = qr0 ? *reinterpret_cast<const uint32_t*>(qr0 + c0 + 8) : 0u;
        qa[kk][3] = qr1 ? *reinterpret_cast<const uint32_t*>(qr1 + c0 + 8) : 0u;
      }
    } else {
      // k16 step kk takes d = 16 (tig + 4 (kk / 4)) + 4 (kk % 4) + {0, 1 | 2, 3}: the
      // four consecutive K bytes this thread reads for that step
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int d0 = 16 * (tig + 4 * (kk >> 2)) + 4 * (kk & 3);
        const uint2 x0 = qr0 ? *reinterpret_cast<const uint2*>(qr0 + d0) : make_uint2(0u, 0u);
        const uint2 x1 = qr1 ? *reinterpret_cast<const uint2*>(qr1 + d0) : make_uint2(0u, 0u);
        qa[kk][0] = bf16x2_to_f16x2(x0.x);
        qa[kk][1] = bf16x2_to_f16x2(x1.x);
        qa[kk][2] = bf16x2_to_f16x2(x0.y);
        qa[kk][3] = bf16x2_to_f16x2(x1.y);
      }
    }
  };

  int at = 0;   // tiles of the segments before
  Segment next;
  if constexpr (SEL) {
    if (p.stream) next = stream_segment<PAGED>(p, plan, x, x1);
    load_q(p.stream ? next.b : b, p.stream ? next.g : g);
  }
  for (;;) {
  if constexpr (SEL) {
    if (p.stream) {
      b = next.b;
      g = next.g;
      tok_begin = next.tok_begin;
      n_tiles = next.n_tiles;
      item = next.item;
      sk = next.sk;
    }
  }
  const int L = sk.L;
  if constexpr (FP8) {
    scale_log2 = p.scale_log2 * __ldg(p.k_scale + g);
    v_scale = __ldg(p.v_scale + g);
  }

  // Query rows r0 = mt*16 + gid and r1 = r0 + 8; row r is (token t = r / G, head g*G + r % G).
  const int r0 = mt * 16 + gid, r1 = r0 + 8;
  int end0 = L, end1 = L;   // first invisible key of each row
  if (p.causal) {
    if (r0 < p.R) end0 = L - p.T + r0 / p.G + 1;
    if (r1 < p.R) end1 = L - p.T + r1 / p.G + 1;
  }
  // SEL: a row sees keys below `sinks` and from its window's first key on; no row sees
  // [sinks, dead_end), whose V rows are zeroed like those past L (they may hold anything)
  const int lo0 = SEL ? end0 - p.sel.window : 0, lo1 = SEL ? end1 - p.sel.window : 0;
  const int dead_end = SEL && p.causal ? L - p.T + 1 - p.sel.window : 0;
  auto dead = [&](int tok) { return tok >= L || (SEL && tok >= p.sel.sinks && tok < dead_end); };
  auto has_dead = [&](int tok0) {   // among tok0 .. tok0 + 15
    return tok0 + 16 > L || (SEL && tok0 < dead_end && tok0 + 16 > p.sel.sinks);
  };

  if constexpr (!SEL) load_q(b, g);

  float o_acc[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o_acc[n][0] = o_acc[n][1] = o_acc[n][2] = o_acc[n][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  // ldmatrix lane roles
  const int lm = lane >> 3, lr = lane & 7;

  for (int i = 0; i < n_tiles; ++i) {
    const int it = SEL ? at + i : i;
    const int s = it % C::kStages;
    if (!mbar_wait(&full[s], (it / C::kStages) & 1)) {
      atomicOr(p.status, DEV_TIMEOUT);
      *reinterpret_cast<volatile int*>(abort_flag) = 1;   // every consumer sees it after the barrier below
      break;
    }
    if (*reinterpret_cast<volatile int*>(abort_flag)) break;
    // SEL: a stage holds block after block of 16 rows, each span of them together
    constexpr int kSpan = SEL ? kPageTokens * 128 : C::kHalfBytes;
    const int block0 = SEL ? wsub * (C::kHalves - 1) * kSpan : 0;
    const uint32_t kbase = smem_u32(smem + s * C::kStageBytes) + block0;
    const uint32_t vbase = kbase + C::kTensorBytes;
    const int tok_base = tok_begin + i * kDecodeTile + wsub * 16;

    // ---- S = Q K^T for this warp's 16 tokens (two n8 tiles)
    float sacc[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) sacc[n][0] = sacc[n][1] = sacc[n][2] = sacc[n][3] = 0.f;
    if constexpr (!FP8) {
      const int trow = wsub * 16 + (lm >> 1) * 8 + lr;   // token row inside the tile
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int chunk16 = kk * 2 + (lm & 1);             // 16-byte chunk along d
        const int h = chunk16 >> 3, cw = chunk16 & 7;
        const uint32_t addr = kbase + h * kSpan + trow * 128 + ((cw ^ (trow & 7)) << 4);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(addr, b0, b1, b2, b3);
        mma_bf16_16816(sacc[0], qa[kk], b0, b1);
        mma_bf16_16816(sacc[1], qa[kk], b2, b3);
      }
    } else {
      // token rows gid (n8 block 0) and 8 + gid (block 1); 16-byte chunks tig and tig + 4
      uint32_t kw[2][8];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const int trow = wsub * 16 + nb * 8 + gid;       // trow & 7 == gid
        const uint32_t ra = kbase + trow * 128;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint4 x = lds128(ra + (((tig + 4 * hh) ^ gid) << 4));
          kw[nb][4 * hh + 0] = x.x;
          kw[nb][4 * hh + 1] = x.y;
          kw[nb][4 * hh + 2] = x.z;
          kw[nb][4 * hh + 3] = x.w;
        }
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          uint32_t b0, b1;
          e4m3x4_to_f16x2x2(kw[nb][kk], b0, b1);
          mma_f16_16816(sacc[nb], qa[kk], b0, b1);
        }
      }
    }

    // ---- V fragments for this warp's 16 tokens, loaded before the softmax so the
    //      shared-memory latency overlaps it; keys at or past L may hold anything
    //      (even NaN), so their V rows are zeroed
    uint32_t vb[FP8 ? 1 : D / 16][4];
    uint32_t vw[FP8 ? 4 : 1][4];   // FP8: 16 bytes (d = 16 gid .. 16 gid + 15) of keys 2tig, 2tig+1, 2tig+8, 2tig+9
    if constexpr (FP8) {
      const bool tail = has_dead(tok_base);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 2 * tig + (i & 1) + 8 * (i >> 1);
        const int vrow = wsub * 16 + key;
        uint4 x = lds128(vbase + vrow * 128 + ((gid ^ (vrow & 7)) << 4));
        if (tail && dead(tok_base + key)) x = make_uint4(0u, 0u, 0u, 0u);
        vw[i][0] = x.x;
        vw[i][1] = x.y;
        vw[i][2] = x.z;
        vw[i][3] = x.w;
      }
    } else {
      const bool tail = has_dead(tok_base);
      const int vrow = wsub * 16 + (lm & 1) * 8 + lr;
      const int ta = tok_base + tig * 2, tb = ta + 8;
      const uint32_t keep_a = (dead(ta) ? 0u : 0x0000ffffu) | (dead(ta + 1) ? 0u : 0xffff0000u);
      const uint32_t keep_b = (dead(tb) ? 0u : 0x0000ffffu) | (dead(tb + 1) ? 0u : 0xffff0000u);
#pragma unroll
      for (int nn = 0; nn < D / 16; ++nn) {
        const int chunk16 = nn * 2 + (lm >> 1);
        const int h = chunk16 >> 3, cw = chunk16 & 7;
        const uint32_t addr = vbase + h * kSpan + vrow * 128 + ((cw ^ (vrow & 7)) << 4);
        ldsm_x4_t(addr, vb[nn][0], vb[nn][1], vb[nn][2], vb[nn][3]);
        if (tail) {
          vb[nn][0] &= keep_a;
          vb[nn][2] &= keep_a;
          vb[nn][1] &= keep_b;
          vb[nn][3] &= keep_b;
        }
      }
    }

    // ---- online softmax (base-2 exponent, scale folded in).  A row's reference
    //      maximum is raised only when the tile maximum exceeds it by more than 8,
    //      so O is rescaled rarely; p = 2^(s - m) then stays <= 256, and the merge
    //      at the end uses the same reference, so the result is exact.
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = tok_base + n * 8 + tig * 2 + (e & 1);
        const int end = (e < 2) ? end0 : end1;
        bool seen = tok < end;
        if constexpr (SEL) seen = seen && (tok >= ((e < 2) ? lo0 : lo1) || tok < p.sel.sinks);
        const float v = seen ? sacc[n][e] * scale_log2 : -INFINITY;
        sacc[n][e] = v;
        if (e < 2) mx0 = fmaxf(mx0, v); else mx1 = fmaxf(mx1, v);
      }
    }
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    if (__any_sync(0xffffffffu, mx0 > m0 + 8.f || mx1 > m1 + 8.f)) {
      const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
      const float al0 = ex2(m0 - ((mn0 == -INFINITY) ? 0.f : mn0));   // 0 while m is -inf
      const float al1 = ex2(m1 - ((mn1 == -INFINITY) ? 0.f : mn1));
      m0 = mn0;
      m1 = mn1;
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o_acc[n][0] *= al0;
        o_acc[n][1] *= al0;
        o_acc[n][2] *= al1;
        o_acc[n][3] *= al1;
      }
    }
    const float mu0 = (m0 == -INFINITY) ? 0.f : m0;
    const float mu1 = (m1 == -INFINITY) ? 0.f : m1;
    float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      sacc[n][0] = ex2(sacc[n][0] - mu0);
      sacc[n][1] = ex2(sacc[n][1] - mu0);
      sacc[n][2] = ex2(sacc[n][2] - mu1);
      sacc[n][3] = ex2(sacc[n][3] - mu1);
      ps0 += sacc[n][0] + sacc[n][1];
      ps1 += sacc[n][2] + sacc[n][3];
    }
    l0 += ps0;
    l1 += ps1;
    uint32_t pa[4];
    if constexpr (!FP8) {
      pa[0] = pack_bf16x2(sacc[0][0], sacc[0][1]);
      pa[1] = pack_bf16x2(sacc[0][2], sacc[0][3]);
      pa[2] = pack_bf16x2(sacc[1][0], sacc[1][1]);
      pa[3] = pack_bf16x2(sacc[1][2], sacc[1][3]);

      // ---- O += P V
#pragma unroll
      for (int nn = 0; nn < D / 16; ++nn) {
        mma_bf16_16816(o_acc[2 * nn], pa, vb[nn][0], vb[nn][1]);
        mma_bf16_16816(o_acc[2 * nn + 1], pa, vb[nn][2], vb[nn][3]);
      }
    } else {
      pa[0] = pack_f16x2(sacc[0][0], sacc[0][1]);
      pa[1] = pack_f16x2(sacc[0][2], sacc[0][3]);
      pa[2] = pack_f16x2(sacc[1][0], sacc[1][1]);
      pa[3] = pack_f16x2(sacc[1][2], sacc[1][3]);
      // ---- O += P V over 16 blocks of 8 output columns; block j, column n is d = 16 n + j,
      //      i.e. byte j of this thread's 16 V bytes; a byte permute pairs keys (2tig, 2tig+1)
      //      and (2tig+8, 2tig+9) for blocks j and j + 1
#pragma unroll
      for (int jj = 0; jj < D / 16; ++jj) {
        const int w = jj >> 1;
        const uint32_t sel = (jj & 1) ? 0x7362u : 0x5140u;
        uint32_t b01_j, b01_j1, b23_j, b23_j1;
        e4m3x4_to_f16x2x2(prmt(vw[0][w], vw[1][w], sel), b01_j, b01_j1);
        e4m3x4_to_f16x2x2(prmt(vw[2][w], vw[3][w], sel), b23_j, b23_j1);
        mma_f16_16816(o_acc[2 * jj], pa, b01_j, b23_j);
        mma_f16_16816(o_acc[2 * jj + 1], pa, b01_j1, b23_j1);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  }

  if constexpr (SEL) {
    // ------------------------------------------------ merge the four warps (the ring goes on)
    constexpr int kC = C::kConsumerWarps * 32;
    if (consumers_abort<kC>(abort_flag)) {
      // a wait gave up: this segment and the rest of the share are left as NaN
      if (p.out.on) {
        p.out.store_nan<D>(b, g, 0, p.R, threadIdx.x, kC);
        return;
      }
      for (;;) {
        for (int r = threadIdx.x; r < p.R; r += kC) p.part_lse[item * p.R + r] = NAN;
        if (!p.stream || (x += n_tiles) >= x1) return;
        const Segment sg = stream_segment<PAGED>(p, plan, x, x1);
        n_tiles = sg.n_tiles;
        item = sg.item;
      }
    }
    at += n_tiles;
    x += n_tiles;
    const bool more = p.stream && x < x1;
    if (more) {   // the next segment's Q is on its way during the merge
      next = stream_segment<PAGED>(p, plan, x, x1);
      load_q(next.b, next.g);
    }
    bool bad = false;
    if (FP8 && p.stream && bad_scale(g)) {
      if (threadIdx.x == 0) atomicOr(p.status, DEV_SCALE);
      bad = true;
    }
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (tig == 0) {
      float* st = stats + ((mt * 4 + wsub) * 16) * 2;
      st[gid * 2 + 0] = m0;
      st[gid * 2 + 1] = l0;
      st[(gid + 8) * 2 + 0] = m1;
      st[(gid + 8) * 2 + 1] = l1;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kC) : "memory");
    float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float* sw = stats + ((mt * 4 + w) * 16) * 2;
      M0 = fmaxf(M0, sw[gid * 2]);
      M1 = fmaxf(M1, sw[(gid + 8) * 2]);
    }
    const float f0 = (m0 == -INFINITY) ? 0.f : ex2(m0 - M0);
    const float f1 = (m1 == -INFINITY) ? 0.f : ex2(m1 - M1);
    // pass ps: rows 4 ps .. 4 ps + 3 of each row group; columns stay in fragment order
    float* merge = reinterpret_cast<float*>(smem + C::kMergeOffset) + mt * 4 * C::kPassRows * C::kMergeStride;
    const int passes = (min(p.R, 16) + C::kPassRows - 1) / C::kPassRows;
#pragma unroll 1
    for (int ps = 0; ps < passes; ++ps) {
      if (ps > 0) asm volatile("bar.sync 1, %0;" ::"n"(kC) : "memory");   // the buffer has been read
      if ((gid >> 2) == (ps & 1)) {
        float* red = merge + (wsub * C::kPassRows + (gid & 3)) * C::kMergeStride + tig * 2;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(red + n * 8) = ps < 2 ? make_float2(o_acc[n][0] * f0, o_acc[n][1] * f0)
                                                           : make_float2(o_acc[n][2] * f1, o_acc[n][3] * f1);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kC) : "memory");
      constexpr int kVec = D / 4;
      const int idx = wsub * 32 + lane, rr = 4 * ps + idx / kVec, r = mt * 16 + rr, v = idx % kVec;
      if (idx < C::kPassRows * kVec && r < p.R) {
        float mrow = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) mrow = fmaxf(mrow, stats[((mt * 4 + w) * 16 + rr) * 2]);
        float lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float mw = stats[((mt * 4 + w) * 16 + rr) * 2];
          const float fw = (mw == -INFINITY) ? 0.f : ex2(mw - mrow);
          lsum += stats[((mt * 4 + w) * 16 + rr) * 2 + 1] * fw;
          const float* src = merge + (w * C::kPassRows + idx / kVec) * C::kMergeStride;
          if constexpr (!FP8) {
            const float4 y = *reinterpret_cast<const float4*>(src + 4 * v);
            acc.x += y.x;
            acc.y += y.y;
            acc.z += y.z;
            acc.w += y.w;
          } else {
            // d = 32 t + n + 16 e stands at 8 n + 2 t + e
            src += (v & 3) * 32 + (v >> 3) * 2 + ((v >> 2) & 1);
            acc.x += src[0];
            acc.y += src[8];
            acc.z += src[16];
            acc.w += src[24];
          }
        }
        const float inv = lsum > 0.f ? (FP8 ? v_scale / lsum : 1.f / lsum) : 0.f;
        const float4 out = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const float lse = bad ? NAN : row_lse(mrow, lsum);
        if (p.out.on) {
          p.out.store4<D>(b, g, r, 4 * v, out);
          if (v == 0) p.out.store_lse(b, g, r, lse);
          continue;
        }
        *reinterpret_cast<float4*>(p.part_o + (item * p.R + r) * (size_t)D + 4 * v) = out;
        if (v == 0) p.part_lse[item * p.R + r] = lse;
      }
    }
    if (!more) break;
  } else {
  // -------------------------------------------------- merge the four warps
  launch_dependents();   // the combine kernel may start launching (it waits for this grid)
  // every consumer reached here; the ring is idle (all issued tiles consumed)
  asm volatile("bar.sync 1, %0;" ::"n"(C::kConsumerWarps * 32) : "memory");
  // one decision for all consumers: a warp that gave up set the shared flag before the
  // barrier, so none of them can wait at a later named barrier for one that left
  if (*reinterpret_cast<volatile int*>(abort_flag)) {
    // a wait gave up: leave the partial as NaN so the result is visibly invalid
    for (int r = threadIdx.x; r < p.R; r += C::kConsumerWarps * 32) p.part_lse[item * p.R + r] = NAN;
    return;
  }
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  float* st = stats + ((mt * 4 + wsub) * 16) * 2;
  if (tig == 0) {
    st[gid * 2 + 0] = m0;
    st[gid * 2 + 1] = l0;
    st[(gid + 8) * 2 + 0] = m1;
    st[(gid + 8) * 2 + 1] = l1;
  }
  asm volatile("bar.sync 1, %0;" ::"n"(C::kConsumerWarps * 32) : "memory");
  float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float* sw = stats + ((mt * 4 + w) * 16) * 2;
    M0 = fmaxf(M0, sw[gid * 2]);
    M1 = fmaxf(M1, sw[(gid + 8) * 2]);
  }
  const float f0 = (m0 == -INFINITY) ? 0.f : ex2(m0 - M0);
  const float f1 = (m1 == -INFINITY) ? 0.f : ex2(m1 - M1);
  float* red = reinterpret_cast<float*>(smem) + ((mt * 4 + wsub) * 16) * C::kRedStride;
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    if constexpr (!FP8) {
      const int col = n * 8 + tig * 2;
      *reinterpret_cast<float2*>(red + gid * C::kRedStride + col) = make_float2(o_acc[n][0] * f0, o_acc[n][1] * f0);
      *reinterpret_cast<float2*>(red + (gid + 8) * C::kRedStride + col) =
          make_float2(o_acc[n][2] * f1, o_acc[n][3] * f1);
    } else {
      const int col = 32 * tig + n;   // columns 2tig and 2tig + 1 of block n are d = 32 tig + n and + 16
      red[gid * C::kRedStride + col] = o_acc[n][0] * f0;
      red[gid * C::kRedStride + col + 16] = o_acc[n][1] * f0;
      red[(gid + 8) * C::kRedStride + col] = o_acc[n][2] * f1;
      red[(gid + 8) * C::kRedStride + col + 16] = o_acc[n][3] * f1;
    }
  }
  asm volatile("bar.sync 1, %0;" ::"n"(C::kConsumerWarps * 32) : "memory");

  float* out = p.part_o + item * (size_t)p.R * D;
  constexpr int kVec = D / 4;   // float4 per row
  for (int idx = threadIdx.x; idx < p.R * kVec; idx += C::kConsumerWarps * 32) {
    const int r = idx / kVec, col = (idx - r * kVec) * 4;
    const int rm = r >> 4, rr = r & 15;
    float mrow = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) mrow = fmaxf(mrow, stats[((rm * 4 + w) * 16 + rr) * 2]);
    float lsum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float mw = stats[((rm * 4 + w) * 16 + rr) * 2];
      const float fw = (mw == -INFINITY) ? 0.f : ex2(mw - mrow);
      lsum += stats[((rm * 4 + w) * 16 + rr) * 2 + 1] * fw;
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) +
                                                        ((rm * 4 + w) * 16 + rr) * C::kRedStride + col);
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    const float inv = lsum > 0.f ? (FP8 ? v_scale / lsum : 1.f / lsum) : 0.f;
    *reinterpret_cast<float4*>(out + (size_t)r * D + col) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (col == 0) p.part_lse[item * p.R + r] = row_lse(mrow, lsum);
  }
  break;
  }
  }
  if (SEL && !p.early) launch_dependents();
}

// kPer consecutive partial-output floats of one lane (2 or 4), as a float4.
template <int kPer>
__device__ __forceinline__ float4 load_part(const float* src) {
  if constexpr (kPer == 4) {
    return __ldg(reinterpret_cast<const float4*>(src));
  } else {
    const float2 v = __ldg(reinterpret_cast<const float2*>(src));
    return make_float4(v.x, v.y, 0.f, 0.f);
  }
}

template <int kPer>
__device__ __forceinline__ void accumulate(float (&acc)[kPer], float w, float4 x) {
  acc[0] = fmaf(w, x.x, acc[0]);
  acc[1] = fmaf(w, x.y, acc[1]);
  if constexpr (kPer == 4) {
    acc[2] = fmaf(w, x.z, acc[2]);
    acc[3] = fmaf(w, x.w, acc[3]);
  }
}

// Merge the chunk partials of each output row (b, t, h).  wpr warps (1, 2, 4 or 8)
// share a row: warp w of the row takes chunks w, w + wpr, ...; their weighted sums
// meet in shared memory.  The sequence length is read before the wait on the split
// kernel (that kernel does not write it); after the wait every warp issues its first
// kBatch partial loads together with the row's LSE loads, so a row costs about two
// dependent memory round trips.  kBatch: partial loads in flight per lane -- 8 for
// long decode (many chunks per row), 2 for launches of at most two chunks (many rows,
// as in a prompt chunk), where a small register footprint buys five CTAs per SM.
// SEL: the sequences' selected keys.  With a shared prefix (pre.chunks > 0) the row's
// first pre.chunks chunks are the prefix's partials.
struct PrefixParts {
  const float* o;
  const float* lse;
  int chunks, rows;     // rows per chunk: B * T * G
  int stream, tiles;    // stream > 0: as in SplitParams, over so many tiles per KV head
};
template <int D, int kBatch, bool SEL>
__global__ void __launch_bounds__(256, kBatch >= 8 ? 2 : 5) decode_combine_kernel(const float* __restrict__ part_o,
                                                             const float* __restrict__ part_lse,
                                                             const int32_t* __restrict__ seqlens, void* o, int o_bf16,
                                                             float* lse, SplitParams p, int B, int paged, int wpr,
                                                             PrefixParts pre) {
  constexpr int kPer = D / 32;    // output columns per lane
  __shared__ float4 red[8][32];   // one float4 per lane of each of the 8 warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wi = warp & (wpr - 1);
  const int row = (blockIdx.x * 8 + warp) / wpr;
  const int rows = B * p.T * p.Hq;
  const bool live = row < rows;
  const int h = row % p.Hq;
  const int t = (row / p.Hq) % p.T;
  const int b = row / (p.Hq * p.T);
  const int g = h / p.G, r = t * p.G + (h - g * p.G);
  bool bad = true;
  int nc = 0, L = 0;
  int before = 0, total = 0;   // p.stream: tiles (per KV head) of the sequences before b, and of all
  if constexpr (SEL) {
    if (p.stream) {
      const int bb = live ? b : 0;
      for (int j = lane; j < B; j += 32) {
        const SeqKeys k = seq_keys<true>(p.sel, seqlens, j, p.T, p.max_seqlen, paged != 0, p.capacity, p.max_blocks);
        const int tiles = k.bad ? 0 : (k.L + kDecodeTile - 1) / kDecodeTile;
        total += tiles;
        if (j < bb) before += tiles;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, off);
        total += __shfl_xor_sync(0xffffffffu, total, off);
      }
    }
  }
  if (live) {
    const SeqKeys sk = seq_keys<SEL>(p.sel, seqlens, b, p.T, p.max_seqlen, paged != 0, p.capacity, p.max_blocks);
    L = sk.L;
    bad = sk.bad;
    if (!bad && !p.balanced && !p.stream) nc = (L + p.chunk - 1) / p.chunk;
  }
  grid_dependency_wait();   // launched early (programmatic dependent launch): the partials are ready after this
  // chunks of this (b, g): fixed length, or the balanced plan the split kernel wrote
  size_t item0 = ((size_t)b * p.Hkv + g) * p.max_chunks;
  if (p.balanced && live && !bad) {
    const int first = p.plan[3 * b], n_b = p.plan[3 * b + 1], chunk_b = p.plan[3 * b + 2];
    nc = (L + chunk_b - 1) / chunk_b;
    item0 = (size_t)p.Hkv * first + (size_t)g * n_b;
  }
  if (SEL && p.stream && live && !bad) {
    const int tiles = (L + kDecodeTile - 1) / kDecodeTile, n = min(p.stream, total);
    const int c0 = stream_cta(before, n, total);
    nc = stream_cta(before + tiles - 1, n, total) - c0 + 1;
    item0 = (size_t)g * (p.stream + B) + c0 + b;
  }
  int npre = 0;
  size_t pre_item0 = 0;
  if constexpr (SEL) {
    if (nc > 0 && pre.o) {
      npre = pre.chunks;
      pre_item0 = (size_t)g * pre.chunks;
      if (pre.stream) {
        npre = min(pre.stream, pre.tiles);
        pre_item0 = (size_t)g * (pre.stream + 1);
      }
    }
  }
  nc += npre;

  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  float lse_row = -INFINITY;
  if (nc > 0) {
    const float* lse0 = part_lse + item0 * p.R + r;            // chunk c at lse0[c * R]
    const float* src0 = part_o + (item0 * p.R + r) * D + lane * kPer;
    const size_t cstride = (size_t)p.R * D;                    // floats between consecutive chunks of this row
    // row of the shared prefix's partials: the whole batch's rows of KV head g, in order
    const size_t pre0 = SEL ? pre_item0 * pre.rows + (size_t)b * p.R + r : 0;
    auto chunk_lse = [&](int c) -> const float* {
      if constexpr (SEL) {
        if (c < npre) return pre.lse + pre0 + (size_t)c * pre.rows;
        c -= npre;
      }
      return lse0 + (size_t)c * p.R;
    };
    auto chunk_o = [&](int c) -> const float* {
      if constexpr (SEL) {
        if (c < npre) return pre.o + (pre0 + (size_t)c * pre.rows) * D + lane * kPer;
        c -= npre;
      }
      return src0 + (size_t)c * cstride;
    };
    const int n0 = min(nc, 32);
    const float lc0 = lane < n0 ? __ldg(chunk_lse(lane)) : -INFINITY;
    float4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int c = wi + u * wpr;
      x[u] = c < n0 ? load_part<kPer>(chunk_o(c)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // log-sum-exp over the chunks: every lane keeps a (max, sum) pair, then the pairs merge
    float m = lc0, sum = lc0 == -INFINITY ? 0.f : 1.f;
    for (int c = 32 + lane; c < nc; c += 32) {
      const float lc = __ldg(chunk_lse(c));
      if (lc == -INFINITY) continue;
      if (!(lc <= m)) {   // NaN too: it stays, whatever m is
        sum = sum * expf(m - lc) + 1.f;
        m = lc;
      } else {
        sum += expf(lc - m);
      }
    }
    float M = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float z = m == -INFINITY ? 0.f : sum * expf(m - M);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    lse_row = M + logf(z);
    // chunk c of the first 32 has its weight on lane c
    const float wl0 = lc0 == -INFINITY ? 0.f : expf(lc0 - lse_row);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int c = wi + u * wpr;
      const float w = __shfl_sync(0xffffffffu, wl0, c & 31);
      if (c < n0) accumulate<kPer>(acc, w, x[u]);
    }
    // what the first batch did not cover: more chunks of the first 32, later groups of 32
    for (int g0 = 0; g0 < nc; g0 += 32) {
      const int n = min(32, nc - g0);
      const int first = g0 == 0 ? wi + kBatch * wpr : wi;
      if (first >= n) continue;
      const float lc = g0 == 0 ? lc0 : (lane < n ? __ldg(chunk_lse(g0 + lane)) : -INFINITY);
      const float wl = lc == -INFINITY ? 0.f : expf(lc - lse_row);
      for (int j0 = first; j0 < n; j0 += kBatch * wpr) {
        float4 y[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = j0 + u * wpr;
          y[u] = j < n ? load_part<kPer>(chunk_o(g0 + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = j0 + u * wpr;
          const float w = __shfl_sync(0xffffffffu, wl, j & 31);
          if (j < n) accumulate<kPer>(acc, w, y[u]);
        }
      }
    }
  }
  if (wpr > 1) {   // the row's warps add up in shared memory; its first warp writes
    if (wi != 0) {
      float4 v = make_float4(acc[0], acc[1], 0.f, 0.f);
      if constexpr (kPer == 4) {
        v.z = acc[2];
        v.w = acc[3];
      }
      red[warp][lane] = v;
    }
    __syncthreads();
    if (wi == 0) {
      for (int k = 1; k < wpr; ++k) {
        const float4 v = red[warp + k][lane];
        acc[0] += v.x;
        acc[1] += v.y;
        if constexpr (kPer == 4) {
          acc[2] += v.z;
          acc[3] += v.w;
        }
      }
    }
  }
  if (!live || wi != 0) return;
  if (bad) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = NAN;
    lse_row = NAN;
  }
  const size_t orow = (((size_t)b * p.T + t) * p.Hq + h) * D + lane * kPer;
  if (o_bf16) {
    __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(o) + orow;
#pragma unroll
    for (int e = 0; e < kPer; e += 2) *reinterpret_cast<__nv_bfloat162*>(ob + e) = __floats2bfloat162_rn(acc[e], acc[e + 1]);
  } else {
    float* of = reinterpret_cast<float*>(o) + orow;
#pragma unroll
    for (int e = 0; e < kPer; ++e) of[e] = acc[e];
  }
  if (lse && lane == 0) lse[((size_t)b * p.Hq + h) * p.T + t] = lse_row;
}

template <int D, int MT, bool PAGED, bool FP8, bool SEL>
cudaError_t run_split_as(const CUtensorMap& tk, const CUtensorMap& tv, const SplitParams& sp, int B,
                      cudaStream_t stream) {
  using C = DecodeCfg<D, MT, FP8>;
  auto kern = decode_split_kernel<D, MT, PAGED, FP8, SEL>;
  constexpr int kSmem = SEL ? C::kSelSmemBytes : C::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  if constexpr (SEL) return launch_sel(kern, C::kThreads, kSmem, tk, tv, sp, B, stream);
  dim3 grid(sp.max_chunks, sp.Hkv, B);
  kern<<<grid, C::kThreads, kSmem, stream>>>(tk, tv, sp);
  return cudaGetLastError();
}

template <int D, int MT, bool PAGED, bool FP8 = false>
cudaError_t run_split(const CUtensorMap& tk, const CUtensorMap& tv, const SplitParams& sp, int B,
                      cudaStream_t stream) {
  return sp.sel.select ? run_split_as<D, MT, PAGED, FP8, true>(tk, tv, sp, B, stream)
                       : run_split_as<D, MT, PAGED, FP8, false>(tk, tv, sp, B, stream);
}

SplitParams split_params(const DecodeLaunch& a) {
  const int G = a.Hq / a.Hkv;
  SplitParams sp;
  sp.q = static_cast<const __nv_bfloat16*>(a.q);
  sp.k_scale = a.k_scale;
  sp.v_scale = a.v_scale;
  sp.seqlens = a.seqlens;
  sp.page_table = a.page_table;
  sp.part_o = a.part_o;
  sp.part_lse = a.part_lse;
  sp.status = a.status;
  sp.T = a.T;
  sp.Hq = a.Hq;
  sp.Hkv = a.Hkv;
  sp.G = G;
  sp.R = G * a.T;
  sp.chunk = a.chunk;
  sp.max_chunks = a.max_chunks;
  sp.capacity = a.capacity;
  sp.max_blocks = a.max_blocks;
  sp.num_blocks = a.num_blocks;
  sp.max_seqlen = a.max_seqlen;
  sp.scale_log2 = a.scale * kLog2e;
  sp.causal = a.causal;
  sp.balanced = a.balanced;
  sp.plan = a.plan;
  sp.sel = a.sel;
  if (a.direct) sp.out = direct_out(a);
  sp.B = a.B;
  sp.stream = a.stream;
  sp.early = a.early;
  sp.fence = a.fence;
  return sp;
}

}  // namespace

namespace {
int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();   // no device here (workspace sizing on a host without one): a B200's 148 SMs
    sms = 148;
  }
  return sms;
}
}  // namespace

int decode_chunk_tokens(int B, int T, int G, int Hkv, int max_seqlen, int num_splits, bool fp8) {
  int chunk;
  if (num_splits > 0) {
    chunk = (int)(((long long)max_seqlen + num_splits - 1) / num_splits);
  } else {
    // Long chunks stream longer and leave fewer partials to merge; short ones
    // balance the grid.  Measured on B200: the warp-MMA kernel (2 CTAs per SM)
    // was best at 2048 tokens for 16 x 8 sequence-heads up to 32K keys and 4096
    // for 8 x 8 up to 128K, i.e. about 14 work items per SM; the FP8 kernel for
    // up to 8 rows (3 CTAs per SM) wants about 21; the tensor-core kernel
    // (2 CTAs per SM) about 9 for row tiles of up to 64 rows and about 4 for full
    // 128-row tiles, whose softmax makes each tile dearer.  Start long and halve
    // until the grid holds that many items (counted as if every sequence had
    // max_seqlen; row tiles of many new tokens count separately).
    const int R = G * T;
    const bool tc = decode_uses_tc(R, fp8);
    const long long units = (long long)B * Hkv * decode_row_tiles(T, G);
    const bool full_tiles = decode_tc_tile_tokens(T, G) * G > 64;
    const long long target = tc ? (full_tiles ? 640 : 1280) : (fp8 && R <= 8 ? 3072 : 2048);
    chunk = tc ? 16384 : 4096;
    while (chunk > 256 && units * (((long long)max_seqlen + chunk - 1) / chunk) < target) chunk >>= 1;
  }
  // a multiple of both kernels' tiles
  chunk = ((chunk + kDecodeTcTile - 1) / kDecodeTcTile) * kDecodeTcTile;
  return chunk < kDecodeTcTile ? kDecodeTcTile : chunk;
}

int prefix_chunk_tokens(int tokens, int G, int Hkv, int prefix, int num_splits, bool fp8) {
  if (num_splits > 0 || !decode_uses_tc(G * tokens, fp8))
    return decode_chunk_tokens(1, tokens, G, Hkv, prefix, num_splits, fp8);
  const long long units = (long long)Hkv * decode_row_tiles(tokens, G);
  // one wave of CTAs: with 64 sequences of 4 heads behind 32K tokens (two row tiles of 8 KV
  // heads), 18 chunks; at 128 chunks their partials alone were 134 MB
  const long long chunks = std::max(kDecodeTcCtasPerSm * device_sms() / units, 1LL);
  const long long chunk = std::max((prefix + chunks - 1) / chunks, 128LL);
  return (int)((chunk + kDecodeTcTile - 1) / kDecodeTcTile * kDecodeTcTile);
}


int decode_balanced_chunks(int B, int Hkv, int items_per_slot) {
  const int n = items_per_slot * kDecodeTcCtasPerSm * device_sms() / Hkv;
  return n > B ? n : B;
}

bool decode_direct(long long units, int max_keys, bool tc) {
  // Times in us, measured on B200: a 64-token tile of a CTA that has its SM to itself (bf16, the
  // heads' rows of a 64-token tile wait for memory, the tensor-core kernel for its own chain of
  // products); with more CTAs than SMs the tiles of two share the SM's bandwidth; and the partials
  // and the combine of a split.  16 x 8 pairs with a window of 1024: 14.5 us a call against 19.7
  // split; 1 x 8 pairs: 11.6 against 8.7.
  // Held against both sides in 108 calls (bf16 at d = 64 and 128, FP8; 4 to 64 rows per KV head; 16,
  // 128 and 320 units; windows of 256, 1024, 4096): within 3 % of the faster one in 72, 10 % in 80.
  // The others are split where whole is faster: more units than two CTAs per SM hold, with windows
  // up to 1024 (320 units, 256 keys: 4 FP8 rows 16.6 us and 9.5 whole, 64 bf16 rows 43.6 and 25.0), and
  // the tensor-core kernel with few units or 1024 keys (16 units, 256 keys, 64 rows: 14.3 and 10.9).
  const double tiles = (max_keys + kDecodeTile - 1) / kDecodeTile, sms = device_sms(), tile = tc ? 1.3 : 0.65;
  const double waves = units <= sms ? 1.0 : 1.7 * ceil(units / (2 * sms));
  return tiles * tile * waves <= tiles * 0.55 * units / sms + 5.0;
}

bool decode_shared_together(int B, int T, int G, int Hkv, int max_seqlen, int prefix, bool fp8) {
  // us on B200, as in decode_direct (0.55 a tile with two CTAs per SM, 1.0 on the tensor-core kernel,
  // 8 to start, split and merge), against the three launches of the shared form: 4 sequences behind
  // 1024 tokens 11.1 us instead of 14.3, 40 behind 256 tokens 8.6 instead of 13.8.  Not on the
  // tensor-core kernel: the lookup there slowed every shared call (94 to 99 us behind 32768 tokens).
  // Held against both sides in 54 calls (bf16 at d = 64 and 128, FP8; 4 and 16 rows per KV head; 4, 12 and
  // 40 sequences behind 256, 1024 and 4096 tokens): within 3 % of the faster one in 43, 12 % in 49; the
  // worst are 4 sequences of 4 rows behind 4096 (20.6 us, read by each 15.5) and of 16 rows behind 1024
  // (20.9, three launches 16.4).
  const int rows = G * T;
  if (decode_uses_tc(rows, fp8)) return false;
  const double sms = device_sms();
  auto share = [&](int rows, int row_tiles, double tiles) {
    return tiles * row_tiles * Hkv * (decode_uses_tc(rows, fp8) ? 1.0 : 0.55) / sms;
  };
  const double all = (double)B * ((max_seqlen + kDecodeTile - 1) / kDecodeTile);
  const double own = (double)B * ((max_seqlen - prefix + kDecodeTile - 1) / kDecodeTile);
  const double pre = (prefix + kDecodeTile - 1) / kDecodeTile;
  return share(rows, 1, all) + 8.0 <
         share(rows, 1, own) + share(rows * B, decode_row_tiles(B * T, G), pre) + 13.0;
}

int decode_stream_ctas(int B, int R, int Hkv, int max_keys, bool fp8) {
  if (B > kStreamMaxB || (long long)B * ((max_keys + kDecodeTile - 1) / kDecodeTile) > INT32_MAX) return 0;
  const int per_sm = fp8 ? (R <= 8 ? 3 : (R <= 16 ? 2 : 1)) : 2;   // resident CTAs of the kernel
  return std::max(per_sm * device_sms() / Hkv, 1);
}

cudaError_t launch_decode_split(const DecodeLaunch& a, cudaStream_t stream) {
  const bool paged = a.page_table != nullptr;
  const int R = a.Hq / a.Hkv * a.T;
  const SplitParams sp = split_params(a);

  // K/V viewed as 3-D {d, Hkv, rows}: rows = B * capacity (contiguous) or num_blocks * 16 (paged)
  const uint64_t rows = paged ? (uint64_t)a.num_blocks * kPageTokens : (uint64_t)a.B * a.capacity;
  const bool tc = decode_uses_tc(R, a.fp8 != 0);
  const uint32_t box_rows = paged || a.sel.select ? kPageTokens : (tc ? kDecodeTcTile : kDecodeTile);
  CUtensorMap tk, tv;
  const int eb = a.fp8 ? 1 : 2;   // bytes per cached element
  const uint64_t s1 = (uint64_t)a.d * eb, s2 = (uint64_t)a.Hkv * a.d * eb;
  const uint32_t box0 = 128 / eb;  // one 128-byte swizzle span
  if (a.sel.select && !tc) {
    // {span, head, row, spans of a row}: one copy takes a block's rows span by span
    const cuuint64_t dims[4] = {box0, (cuuint64_t)a.Hkv, rows, (cuuint64_t)(s1 / 128)};
    const cuuint64_t strides[3] = {s1, s2, 128};
    const cuuint32_t box[4] = {box0, 1, (cuuint32_t)kPageTokens, (cuuint32_t)(s1 / 128)};
    if (encode_tmap_nd(&tk, a.k, 4, dims, strides, box, eb) || encode_tmap_nd(&tv, a.v, 4, dims, strides, box, eb))
      return cudaErrorInvalidValue;
  } else if (encode_tmap_3d(&tk, a.k, a.d, a.Hkv, rows, s1, s2, box0, 1, box_rows, eb) ||
      encode_tmap_3d(&tv, a.v, a.d, a.Hkv, rows, s1, s2, box0, 1, box_rows, eb))
    return cudaErrorInvalidValue;

  cudaError_t e;
  if (tc) {
    e = launch_decode_tc(a, tk, tv, stream);   // bf16 above 16 rows per KV head, FP8 above 32
  } else if (a.sel.select && R <= 8) {
    e = launch_decode_rows8(tk, tv, sp, a.B, a.d, a.fp8 != 0, paged, stream);
  } else if (a.fp8) {
    // api.cu admits FP8 caches with d == 128 only
    if (R <= 8) e = launch_decode_fp8_rows8(tk, tv, sp, a.B, paged, stream);
    else if (R <= 16) e = paged ? run_split<128, 1, true, true>(tk, tv, sp, a.B, stream)
                           : run_split<128, 1, false, true>(tk, tv, sp, a.B, stream);
    else e = paged ? run_split<128, 2, true, true>(tk, tv, sp, a.B, stream)
                   : run_split<128, 2, false, true>(tk, tv, sp, a.B, stream);
  } else if (a.d == 128) {   // at most kDecodeMmaRows (16) rows: one row group
    e = paged ? run_split<128, 1, true>(tk, tv, sp, a.B, stream) : run_split<128, 1, false>(tk, tv, sp, a.B, stream);
  } else {
    e = paged ? run_split<64, 1, true>(tk, tv, sp, a.B, stream) : run_split<64, 1, false>(tk, tv, sp, a.B, stream);
  }
  return e;
}

cudaError_t launch_decode(const DecodeLaunch& a, cudaStream_t stream) {
  const cudaError_t e = launch_decode_split(a, stream);
  return e != cudaSuccess || a.direct ? e : launch_decode_combine(a, stream);
}

cudaError_t launch_decode_combine(const DecodeLaunch& a, cudaStream_t stream) {
  const SplitParams sp = split_params(a);

  // the combine kernel is launched as a programmatic dependent of the split kernel:
  // it starts launching while the split kernel's last CTAs finish and waits for them
  // warps per output row: enough that each warp merges at most four chunks
  int wpr = 1;
  int row_chunks = sp.max_chunks + a.pre_chunks;
  if (a.sel.select) {
    // the chunks that a row has when the batch's sequences are of one length
    auto share = [](int n, int units) { return (n + units - 1) / units + 1; };
    row_chunks = sp.stream ? share(sp.stream, a.B) : (a.balanced ? share(a.n_chunks, a.B) : sp.max_chunks);
    if (a.pre_o) row_chunks += a.pre_stream ? std::min(a.pre_stream, a.pre_tiles) : a.pre_chunks;
  }
  const long long rows_out = (long long)a.B * a.T * a.Hq;
  // SEL, many rows: as few waves of CTAs (2 x 8 warps per SM) as possible.  2048 rows of 23
  // chunks took 29 us with 8 warps a row, seven waves that each wait for their loads
  const long long warps = a.sel.select ? 16LL * device_sms() : INT64_MAX;
  while (wpr < 8 && wpr * 4 < row_chunks && rows_out * wpr * 2 <= warps) wpr *= 2;
  const dim3 grid((unsigned)((rows_out * wpr + 7) / 8));
  const int paged_i = a.page_table != nullptr ? 1 : 0;
  const bool light = row_chunks <= 2;
  const PrefixParts pre = {a.pre_o, a.pre_lse, a.pre_chunks, a.B * sp.R, a.pre_stream, a.pre_tiles};
  auto pick = [&](auto sel) {
    constexpr bool S = decltype(sel)::value;
    return a.d == 128 ? (light ? decode_combine_kernel<128, 2, S> : decode_combine_kernel<128, 8, S>)
                      : (light ? decode_combine_kernel<64, 2, S> : decode_combine_kernel<64, 8, S>);
  };
  auto kern = a.sel.select ? pick(std::true_type{}) : pick(std::false_type{});
  return launch_beside(kern, grid, 256, 0, stream, (const float*)a.part_o, (const float*)a.part_lse, a.seqlens, a.o,
                       a.o_bf16, a.lse, sp, a.B, paged_i, wpr, pre);
}

}  // namespace kvattn
