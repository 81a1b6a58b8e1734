// Windowed and shared-prefix decode for at most 8 query rows per KV head, bf16 and FP8
// caches (one new token of up to eight query heads per KV head, two of four, ...).
//
// The products are taken transposed, keys on the MMA's 16 rows and query rows on its 8
// columns: S^T = K Q^T, O^T += V^T P^T.  With the query rows on the 16 rows (decode.cu)
// half of every MMA multiplies zeros: there a 64-token tile took a CTA 1.08 us with two
// CTAs per SM, 9 TB/s at most and less with everything else, and the tile rate, not HBM,
// set the time.
//
// Launch: p.stream CTAs with even shares of the tiles (split.cuh), or one CTA per chunk.
// A producer warp fills a ring of 64-token K/V tiles by TMA; each of four consumer warps
// owns 16 tokens of every tile and keeps its own online softmax; at the end of a segment
// the four are merged and its normalised output and log-sum-exp written, while the ring
// goes on filling with the next one.
//
// A row's reference maximum is raised only when a score exceeds it by more than 8 (base
// 2), so p <= 256 and the result is exact; whether any score does is one vote, and the
// maximum over the keys (three shuffles a row) is taken only then.  16 tokens that every
// row sees skip the masks.
//
// bf16: K and V^T fragments come from shared memory by ldmatrix, P is rounded to bf16
// (half a step, 2^-8 relative, while its sum stays in fp32).  FP8: e4m3 codes become f16
// exactly, the d positions of the K product in the order of the bytes a thread reads and
// the output columns in that of its V bytes (as in decode_fp8.cu); P is rounded to f16
// (2^-11); the K scale is folded into the exponent, the V scale into the normalisation.
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "split.cuh"

namespace kvattn {
namespace {

template <int D, bool FP8>
struct Rows8Cfg {
  static_assert(!FP8 || D == 128, "FP8 caches are built for d = 128");
  static constexpr int kConsumerWarps = 4;
  static constexpr int kThreads = 32 * (kConsumerWarps + 1);
  static constexpr int kRows = 8;                            // query rows per KV head (MMA N)
  static constexpr int kHalves = (FP8 ? D : 2 * D) / 128;    // 128-byte swizzle spans per token row
  static constexpr int kHalfBytes = kDecodeTile * 128;
  static constexpr int kTensorBytes = kHalves * kHalfBytes;  // one of K or V per stage
  static constexpr int kStageBytes = 2 * kTensorBytes;
  static constexpr int kCtasPerSm = FP8 ? 3 : 2;
  static constexpr int kStages = FP8 ? 4 : (D == 128 ? 3 : 6);
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kStatsOffset = kBarOffset + 2 * kStages * 8;        // [4 warps][8 rows][2]: m, l
  static constexpr int kFlagOffset = kStatsOffset + kConsumerWarps * kRows * 2 * 4;
  // merge buffer: four rows of each warp at a time
  static constexpr int kPassRows = 4;
  static constexpr int kMergeStride = D + 4;
  static constexpr int kMergeOffset = (kFlagOffset + 4 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kMergeOffset + kConsumerWarps * kPassRows * kMergeStride * 4 + 1024;
  static_assert(kCtasPerSm * (kSmemBytes + (int)sizeof(StreamPlan) + 1024) <= 228 * 1024, "resident CTAs");
};

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v) {
  return pack_f16x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <int D, bool PAGED, bool FP8>
__global__ void __launch_bounds__(Rows8Cfg<D, FP8>::kThreads, Rows8Cfg<D, FP8>::kCtasPerSm)
    decode_rows8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const SplitParams p) {
  using C = Rows8Cfg<D, FP8>;
  constexpr int kC = C::kConsumerWarps * 32;
  constexpr int kSpan = kPageTokens * 128;   // a 128-byte span of a block's 16 rows
  extern __shared__ uint8_t smem_raw[];
  __shared__ StreamPlan plan;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + C::kStages;
  float* stats = reinterpret_cast<float*>(smem + C::kStatsOffset);
  int* abort_flag = reinterpret_cast<int*>(smem + C::kFlagOffset);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x;

  if (threadIdx.x == kC) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::kConsumerWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (!p.fence) grid_dependency_wait();   // launched early too; with p.fence the kernel before has waited
  if (p.early) launch_dependents();
  if (p.fence && c == (p.stream ? p.stream * p.Hkv : p.max_chunks)) {
    if (blockIdx.y == 0 && blockIdx.z == 0) grid_dependency_wait();
    return;
  }
  int x = 0, x1 = 0;   // p.stream: this CTA's share of the tiles
  Segment sg;
  if (p.stream) {
    if (warp == C::kConsumerWarps) stream_plan<PAGED, C::kThreads>(p, &plan);
    else stream_plan_wait<C::kThreads>();
    const int total = plan.first[p.B], n = min(p.stream, total), i = c / p.Hkv;
    if (i >= n) return;
    x = stream_begin(i, n, total);
    x1 = stream_begin(i + 1, n, total);
    sg = stream_segment<PAGED>(p, &plan, x, x1);
  } else {
    sg.g = blockIdx.y;
    sg.b = blockIdx.z;
    sg.sk = seq_keys<true>(p.sel, p.seqlens, sg.b, p.T, p.max_seqlen, PAGED, p.capacity, p.max_blocks);
    if (sg.sk.bad) {
      if (threadIdx.x == 0 && c == 0 && sg.g == 0) atomicOr(p.status, DEV_SEQLEN);
      if (p.out.on) p.out.store_nan<D>(sg.b, sg.g, 0, p.R, threadIdx.x, blockDim.x);
      return;   // else the combine kernel writes NaN rows for this sequence
    }
    sg.tok_begin = c * p.chunk;
    if (sg.tok_begin >= sg.sk.L) return;
    sg.tok_end = min(sg.tok_begin + p.chunk, sg.sk.L);
    sg.n_tiles = (sg.tok_end - sg.tok_begin + kDecodeTile - 1) / kDecodeTile;
    sg.item = ((size_t)sg.b * p.Hkv + sg.g) * p.max_chunks + c;
    __syncthreads();
  }

  if (warp == C::kConsumerWarps) {
    auto produce = [&](auto prefix) {
      constexpr bool PREFIX = decltype(prefix)::value;
      if (p.stream) {
        produce_stream<C, PAGED, PREFIX>(smem, full, empty, &tmK, &tmV, p, &plan, sg, x, x1, abort_flag);
      } else if (lane == 0) {
        produce_split_tiles<C, PAGED, true, PREFIX>(smem, full, empty, &tmK, &tmV, p, sg.b, sg.g, sg.tok_begin,
                                                    sg.tok_end, sg.n_tiles, sg.sk, abort_flag);
      }
    };
    if (PAGED && p.sel.prefix_blocks) produce(std::bool_constant<PAGED>{});
    else produce(std::false_type{});
    return;
  }

  // -------------------------------------------------------------- consumers
  const int wsub = warp;                       // which 16 tokens of each tile
  const int gid = lane >> 2, tig = lane & 3;
  const int lm = lane >> 3, lr = lane & 7;     // ldmatrix roles: matrix and row
  const int r0 = 2 * tig, r1 = r0 + 1;         // this thread's S^T columns: query rows t * G + head of the group

  // Q^T (B operand, n = query row gid).  FP8: k16 step kk takes
  // d = 16 (tig + 4 (kk / 4)) + 4 (kk % 4) + {0, 1 | 2, 3}
  uint32_t qb[D / 16][2];
  auto load_q = [&](int b, int g) {
    const int t = gid / p.G, hh = gid - t * p.G;
    const __nv_bfloat16* qr = p.q + (((size_t)b * p.T + t) * p.Hq + (size_t)g * p.G + hh) * D;
    const bool live = gid < p.R;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      if constexpr (FP8) {
        const int d0 = 16 * (tig + 4 * (kk >> 2)) + 4 * (kk & 3);
        const uint2 v = live ? *reinterpret_cast<const uint2*>(qr + d0) : make_uint2(0u, 0u);
        qb[kk][0] = bf16x2_to_f16x2(v.x);
        qb[kk][1] = bf16x2_to_f16x2(v.y);
      } else {
        qb[kk][0] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + tig * 2) : 0u;
        qb[kk][1] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + tig * 2 + 8) : 0u;
      }
    }
  };
  load_q(sg.b, sg.g);

  int at = 0;   // tiles of the segments before
  for (;;) {
    const int L = sg.sk.L;
    float scale_log2 = p.scale_log2, v_scale = 1.f;
    bool bad = false;
    if constexpr (FP8) {
      const float ks = __ldg(p.k_scale + sg.g);
      v_scale = __ldg(p.v_scale + sg.g);
      bad = !(ks > 0.f && ks <= 3.402823466e38f && v_scale > 0.f && v_scale <= 3.402823466e38f);
      if (bad && threadIdx.x == 0) atomicOr(p.status, DEV_SCALE);
      scale_log2 *= ks;
    }
    // rows see keys below their end, from their window's first key on or among the first
    // `sinks`; rows past the last live one are computed and dropped
    const int first_end = p.causal ? L - p.T + 1 : L;
    const int end0 = p.causal && r0 < p.R ? first_end + r0 / p.G : L;
    const int end1 = p.causal && r1 < p.R ? first_end + r1 / p.G : L;
    const int lo0 = end0 - p.sel.window, lo1 = end1 - p.sel.window, last_lo = L - p.sel.window;
    // no row sees [sinks, dead_end) or [L, ...): those V rows may hold anything and are zeroed
    const int dead_end = first_end - p.sel.window;
    auto seen = [&](int tok, int end, int lo) { return tok < end && (tok >= lo || tok < p.sel.sinks); };
    auto dead = [&](int tok) { return tok >= L || (tok >= p.sel.sinks && tok < dead_end); };

    float o[D / 16][4];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int i = 0; i < sg.n_tiles; ++i) {
      const int it = at + i;
      const int s = it % C::kStages;
      if (!mbar_wait(&full[s], (it / C::kStages) & 1)) {
        atomicOr(p.status, DEV_TIMEOUT);
        *reinterpret_cast<volatile int*>(abort_flag) = 1;   // every consumer learns of it at the segment's end
        break;
      }
      if (*reinterpret_cast<volatile int*>(abort_flag)) break;
      // this warp's 16 tokens: C::kHalves spans of 16 rows
      const uint32_t kbase = smem_u32(smem + s * C::kStageBytes) + wsub * (C::kHalves * kSpan);
      const uint32_t vbase = kbase + C::kTensorBytes;
      const int tok_base = sg.tok_begin + i * kDecodeTile + wsub * 16;
      const bool inside = tok_base + 16 <= first_end && (tok_base >= last_lo || tok_base + 16 <= p.sel.sinks);

      // ---- S^T = K Q^T, in two chains
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (FP8) {
        // A rows are keys gid and gid + 8 of this warp's 16 (token row & 7 == gid)
        uint32_t kw[2][8];
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const uint32_t ra = kbase + (rr * 8 + gid) * 128;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint4 w = lds128(ra + (((tig + 4 * hh) ^ gid) << 4));
            kw[rr][4 * hh + 0] = w.x;
            kw[rr][4 * hh + 1] = w.y;
            kw[rr][4 * hh + 2] = w.z;
            kw[rr][4 * hh + 3] = w.w;
          }
        }
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t a[4];
          e4m3x4_to_f16x2x2(kw[0][kk], a[0], a[2]);
          e4m3x4_to_f16x2x2(kw[1][kk], a[1], a[3]);
          mma_f16_16816((kk & 1) ? sb : sa, a, qb[kk][0], qb[kk][1]);
        }
      } else {
        const int trow = (lm & 1) * 8 + lr;   // key; matrices 2 and 3 are the next 16 bytes of d
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int chunk16 = kk * 2 + (lm >> 1);
          const int h = chunk16 >> 3, cw = chunk16 & 7;
          uint32_t a[4];
          ldsm_x4(kbase + h * kSpan + trow * 128 + ((cw ^ (trow & 7)) << 4), a[0], a[1], a[2], a[3]);
          mma_bf16_16816((kk & 1) ? sb : sa, a, qb[kk][0], qb[kk][1]);
        }
      }

      // ---- V of this warp's 16 tokens, loaded before the softmax so the latency overlaps it
      uint32_t vw[FP8 ? 4 : D / 16][4];
      if constexpr (FP8) {
        // bytes d = 16 gid .. 16 gid + 15 of keys 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int key = 2 * tig + (q & 1) + 8 * (q >> 1);
          uint4 w = lds128(vbase + key * 128 + ((gid ^ (key & 7)) << 4));
          if (!inside && dead(tok_base + key)) w = make_uint4(0u, 0u, 0u, 0u);
          vw[q][0] = w.x;
          vw[q][1] = w.y;
          vw[q][2] = w.z;
          vw[q][3] = w.w;
        }
      } else {
        // V^T fragments: matrices (keys 0-7 | 8-15) x (d 0-7 | 8-15), transposed on the way
        const int vrow = (lm >> 1) * 8 + lr;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const int chunk16 = j * 2 + (lm & 1);
          const int h = chunk16 >> 3, cw = chunk16 & 7;
          ldsm_x4_t(vbase + h * kSpan + vrow * 128 + ((cw ^ (vrow & 7)) << 4), vw[j][0], vw[j][1], vw[j][2],
                    vw[j][3]);
        }
        if (!inside) {
          const int ta = tok_base + tig * 2, tb = ta + 8;
          const uint32_t keep_a = (dead(ta) ? 0u : 0x0000ffffu) | (dead(ta + 1) ? 0u : 0xffff0000u);
          const uint32_t keep_b = (dead(tb) ? 0u : 0x0000ffffu) | (dead(tb + 1) ? 0u : 0xffff0000u);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            vw[j][0] &= keep_a;
            vw[j][1] &= keep_a;
            vw[j][2] &= keep_b;
            vw[j][3] &= keep_b;
          }
        }
      }

      // ---- online softmax over this warp's keys for query rows r0, r1
      float v00 = (sa[0] + sb[0]) * scale_log2, v01 = (sa[1] + sb[1]) * scale_log2;   // key gid
      float v10 = (sa[2] + sb[2]) * scale_log2, v11 = (sa[3] + sb[3]) * scale_log2;   // key gid + 8
      if (!inside) {
        const int ka = tok_base + gid, kb = ka + 8;
        v00 = seen(ka, end0, lo0) ? v00 : -INFINITY;
        v01 = seen(ka, end1, lo1) ? v01 : -INFINITY;
        v10 = seen(kb, end0, lo0) ? v10 : -INFINITY;
        v11 = seen(kb, end1, lo1) ? v11 : -INFINITY;
      }
      float mx0 = fmaxf(v00, v10), mx1 = fmaxf(v01, v11);
      if (__any_sync(0xffffffffu, mx0 > m0 + 8.f || mx1 > m1 + 8.f)) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
        }
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        const float al0 = ex2(m0 - ((mn0 == -INFINITY) ? 0.f : mn0));   // 0 while m is -inf
        const float al1 = ex2(m1 - ((mn1 == -INFINITY) ? 0.f : mn1));
        m0 = mn0;
        m1 = mn1;
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[j][0] *= al0;
          o[j][2] *= al0;
          o[j][1] *= al1;
          o[j][3] *= al1;
        }
      }
      const float mu0 = (m0 == -INFINITY) ? 0.f : m0;
      const float mu1 = (m1 == -INFINITY) ? 0.f : m1;
      const float p00 = ex2(v00 - mu0), p10 = ex2(v10 - mu0);
      const float p01 = ex2(v01 - mu1), p11 = ex2(v11 - mu1);
      l0 += p00 + p10;
      l1 += p01 + p11;
      // P^T as the B operand: transpose the 8x8 (key, row) fragments of keys 0-7 and 8-15
      const uint32_t pb0 = movmatrix_trans(FP8 ? pack_f16x2(p00, p01) : pack_bf16x2(p00, p01));
      const uint32_t pb1 = movmatrix_trans(FP8 ? pack_f16x2(p10, p11) : pack_bf16x2(p10, p11));

      // ---- O^T += V^T P^T, blocks of 16 output columns.  bf16: row m of block j is d = 16 j + m.
      //      FP8: d = 16 (m mod 8) + 2 j + (m >= 8), bytes 2j and 2j + 1 of the thread's V chunk,
      //      paired across keys by a byte permute
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        if constexpr (FP8) {
          const int w = j >> 1;
          const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
          uint32_t a[4];
          e4m3x4_to_f16x2x2(prmt(vw[0][w], vw[1][w], sel), a[0], a[1]);
          e4m3x4_to_f16x2x2(prmt(vw[2][w], vw[3][w], sel), a[2], a[3]);
          mma_f16_16816(o[j], a, pb0, pb1);
        } else {
          mma_bf16_16816(o[j], vw[j], pb0, pb1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ------------------------------------------------ merge the four warps (the ring goes on)
    if (consumers_abort<kC>(abort_flag)) {
      // a wait gave up: this segment and the rest of the share are left as NaN
      if (p.out.on) {
        p.out.store_nan<D>(sg.b, sg.g, 0, p.R, threadIdx.x, kC);
        return;
      }
      for (;;) {
        for (int r = threadIdx.x; r < p.R; r += kC) p.part_lse[sg.item * p.R + r] = NAN;
        if (!p.stream || (x += sg.n_tiles) >= x1) return;
        sg = stream_segment<PAGED>(p, &plan, x, x1);
      }
    }
    at += sg.n_tiles;
    x += sg.n_tiles;
    const size_t item = sg.item;
    const bool more = p.stream && x < x1;
    if (more) {   // the next segment's Q is on its way during the merge
      sg = stream_segment<PAGED>(p, &plan, x, x1);
      load_q(sg.b, sg.g);
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (gid == 0) {
      float* st = stats + wsub * C::kRows * 2;
      st[r0 * 2 + 0] = m0;
      st[r0 * 2 + 1] = l0;
      st[r1 * 2 + 0] = m1;
      st[r1 * 2 + 1] = l1;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kC) : "memory");
    float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < C::kConsumerWarps; ++w) {
      M0 = fmaxf(M0, stats[(w * C::kRows + r0) * 2]);
      M1 = fmaxf(M1, stats[(w * C::kRows + r1) * 2]);
    }
    const float f0 = (m0 == -INFINITY) ? 0.f : ex2(m0 - M0);
    const float f1 = (m1 == -INFINITY) ? 0.f : ex2(m1 - M1);
    float* merge = reinterpret_cast<float*>(smem + C::kMergeOffset);
    const int passes = (p.R + C::kPassRows - 1) / C::kPassRows;
#pragma unroll 1
    for (int ps = 0; ps < passes; ++ps) {   // rows 4 ps .. 4 ps + 3
      if (ps > 0) asm volatile("bar.sync 1, %0;" ::"n"(kC) : "memory");   // the buffer has been read
      if ((tig >> 1) == ps) {
        float* red = merge + (wsub * C::kPassRows + (r0 & 3)) * C::kMergeStride;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          if constexpr (FP8) {   // column d = 16 n + 2 j + e stands at 16 j + 2 n + e
            *reinterpret_cast<float2*>(red + 16 * j + 2 * gid) = make_float2(o[j][0] * f0, o[j][2] * f0);
            *reinterpret_cast<float2*>(red + C::kMergeStride + 16 * j + 2 * gid) =
                make_float2(o[j][1] * f1, o[j][3] * f1);
          } else {
            red[16 * j + gid] = o[j][0] * f0;
            red[16 * j + gid + 8] = o[j][2] * f0;
            red[C::kMergeStride + 16 * j + gid] = o[j][1] * f1;
            red[C::kMergeStride + 16 * j + gid + 8] = o[j][3] * f1;
          }
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kC) : "memory");
      const int r = 4 * ps + wsub, v = lane;   // one row per warp, four columns per lane
      if (r < p.R && v < D / 4) {
        float mrow = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::kConsumerWarps; ++w) mrow = fmaxf(mrow, stats[(w * C::kRows + r) * 2]);
        float lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kConsumerWarps; ++w) {
          const float mw = stats[(w * C::kRows + r) * 2];
          const float fw = (mw == -INFINITY) ? 0.f : ex2(mw - mrow);
          lsum += stats[(w * C::kRows + r) * 2 + 1] * fw;
          const float* src = merge + (w * C::kPassRows + wsub) * C::kMergeStride;
          float4 y;
          if constexpr (FP8) {
            src += (v & 3) * 32 + (v >> 2) * 2;
            const float2 y0 = *reinterpret_cast<const float2*>(src), y1 = *reinterpret_cast<const float2*>(src + 16);
            y = make_float4(y0.x, y0.y, y1.x, y1.y);
          } else {
            y = *reinterpret_cast<const float4*>(src + 4 * v);
          }
          acc.x += y.x;
          acc.y += y.y;
          acc.z += y.z;
          acc.w += y.w;
        }
        const float inv = lsum > 0.f ? (FP8 ? v_scale / lsum : 1.f / lsum) : 0.f;
        const float4 out = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const float lse = bad ? NAN : row_lse(mrow, lsum);
        if (p.out.on) {   // sg is still this segment
          p.out.store4<D>(sg.b, sg.g, r, 4 * v, bad ? make_float4(NAN, NAN, NAN, NAN) : out);
          if (v == 0) p.out.store_lse(sg.b, sg.g, r, lse);
          continue;
        }
        *reinterpret_cast<float4*>(p.part_o + (item * p.R + r) * (size_t)D + 4 * v) = out;
        if (v == 0) p.part_lse[item * p.R + r] = lse;
      }
    }
    if (!more) break;
  }
  if (!p.early) launch_dependents();   // the combine kernel may start launching (it waits for this grid)
}

template <int D, bool PAGED, bool FP8>
cudaError_t run(const CUtensorMap& tk, const CUtensorMap& tv, const SplitParams& sp, int B, cudaStream_t stream) {
  using C = Rows8Cfg<D, FP8>;
  auto kern = decode_rows8_kernel<D, PAGED, FP8>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  return e != cudaSuccess ? e : launch_sel(kern, C::kThreads, C::kSmemBytes, tk, tv, sp, B, stream);
}

}  // namespace

cudaError_t launch_decode_rows8(const CUtensorMap& tk, const CUtensorMap& tv, const SplitParams& sp, int B, int d,
                                bool fp8, bool paged, cudaStream_t stream) {
  if (fp8) return paged ? run<128, true, true>(tk, tv, sp, B, stream) : run<128, false, true>(tk, tv, sp, B, stream);
  if (d == 128) return paged ? run<128, true, false>(tk, tv, sp, B, stream) : run<128, false, false>(tk, tv, sp, B, stream);
  return paged ? run<64, true, false>(tk, tv, sp, B, stream) : run<64, false, false>(tk, tv, sp, B, stream);
}

}  // namespace kvattn
