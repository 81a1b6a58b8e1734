// Pieces shared by the split-KV decode kernels (decode.cu, decode_fp8.cu): the
// launch parameters, the length check, the selection of keys, and the TMA producer
// loop that streams a work item's 64-token K/V tiles into a shared-memory ring.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace kvattn {

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
    k.bad = seqlen_bad(k.L, T, max_seqlen, paged, capacity, max_blocks) || k.L - sel.skip < T;
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

// One thread: tiles 0 .. n_tiles-1 of keys [tok_begin, tok_end) into the ring of
// C::kStages stages (K then V, C::kHalves 128-byte swizzle spans per token row;
// contiguous: one 64-row box per span; paged: one 16-row box per physical
// block, its page-table entry bounds-checked first; SEL instances: one 16-row box per
// selected block in either layout), evict-first L2 policy.  A
// stage is refilled once the consumers released it (empty barrier); a wait that
// gives up sets DEV_TIMEOUT and the abort flag.
template <class C, bool PAGED, bool SEL>
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
          ids[j] = j < nb ? (PAGED ? __ldg(row_tab + pos / kPageTokens) : b * p.capacity + pos) : 0;
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
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
          tma_load_3d(kst + h * C::kHalfBytes + j * kPageTokens * 128, tmK, &full[s], h * 64, g, row, pol);
          tma_load_3d(vst + h * C::kHalfBytes + j * kPageTokens * 128, tmV, &full[s], h * 64, g, row, pol);
        }
      }
    }
  }
}

// FP8 caches, at most 8 query rows per KV head: the transposed-product split kernel (decode_fp8.cu)
cudaError_t launch_decode_fp8_rows8(const CUtensorMap& tk, const CUtensorMap& tv, const SplitParams& sp, int B,
                                    bool paged, bool sel, cudaStream_t stream);

}  // namespace kvattn
