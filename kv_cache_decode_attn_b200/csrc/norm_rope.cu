// Per-head RMS norm of queries and keys, the position rotation, and the write of the
// new tokens' K and V, in one pass.
//
// For the row x (d values) of one head of the token at position p:
//   y_i = x_i * rsqrt(mean_j x_j^2 + eps) * w_i            (no weight: y = x)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)    for the rot / 2 pairs
// with pairs (i, i + rot / 2), or (2i, 2i + 1) when interleaved, and the angle table's
// row p holding rot / 2 cosines, then rot / 2 sines.  Values are computed in fp32 and
// rounded once, to bf16 or (FP8 caches) to the e4m3 code of y / scale: rounding to bf16
// between the norm and the rotation, as separate passes do, would only add an error.
//
// d / 16 threads share a row, 16 values each, chosen so that a thread holds both
// members of each of its pairs: only the sum of squares crosses threads (2 or 3
// shuffles).  A warp takes the same 4 (d = 128) or 8 heads of kTokens consecutive tokens,
// all of whose loads go out first; meanwhile the CTA fetches the tokens' angle rows and
// cache rows into shared memory, once for all heads; the weights are unpacked once, and
// values are computed in pairs (f32x2).
// 4 x 4096 tokens of 32 + 8 + 8 heads (405 MB; 62 us at the copy rate): 93 us with one
// token per warp, indexes divided out per row and single fp32 operations (issue slots
// 72 % busy); 98 with the angles read per token by each warp (waiting for them);
// 80 as it is, with three CTAs per SM (99 without that bound on the registers); 81 to 87
// from one B200 to another.
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace kvattn {
namespace {

// Two fp32 values in one register pair.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 parts(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 neg2(F2 a) { return a ^ 0x8000000080000000ull; }

// 8 values, as 4 pairs of neighbours
__device__ __forceinline__ void unpack8(uint4 u, F2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ void load8f(const float* src, F2 (&x)[4]) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  x[0] = f2(a.x, a.y);
  x[1] = f2(a.z, a.w);
  x[2] = f2(b.x, b.y);
  x[3] = f2(b.z, b.w);
}

__device__ __forceinline__ void store8(__nv_bfloat16* dst, const F2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = parts(x[i]);
    w[i] = pack_bf16x2(v.x, v.y);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// codes of x / s, each quotient one IEEE division
__device__ __forceinline__ void store8_e4m3(uint8_t* dst, const F2 (&x)[4], float s) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = parts(x[i]);
    c[i] = f32x2_to_e4m3x2(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s));
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// head_blocks: CTAs per token group, each with blockDim / 32 groups of heads
template <int D, int kTokens, bool CACHED, bool FP8>
__global__ void __launch_bounds__(256, 3) norm_rope_kernel(const NormRopeLaunch a, int head_blocks) {
  constexpr int kLanes = D / 16;       // threads per row
  constexpr int kHeads = 32 / kLanes;  // rows (heads of one token) per warp
  __shared__ __align__(16) float angles[kTokens][D];         // rot / 2 cosines, then rot / 2 sines
  __shared__ long long cache_row[kTokens];     // CACHED: row of the token in the [rows, Hkv, D] view, or -1
  __shared__ int in_table[kTokens];            // whether the position is in the angle table
  const int tg = blockIdx.x / head_blocks;
  const int lane = threadIdx.x & 31, j = lane & (kLanes - 1);
  const int row = ((blockIdx.x - tg * head_blocks) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kHeads + lane / kLanes;
  const bool live = row < a.Hq + a.Hkv * (CACHED ? 2 : 1);        // q heads, K heads, V heads
  const int h = live ? row : 0;
  const bool is_q = h < a.Hq, is_v = CACHED && h >= a.Hq + a.Hkv;
  const int g = is_q ? h : (is_v ? h - a.Hq - a.Hkv : h - a.Hq);   // head among its kind
  const int tok0 = tg * kTokens;
  const int n_tok = min(kTokens, a.B * a.T - tok0);

  // this thread's two vectors of 8 values: both halves of its rotated pairs, or (past the
  // rotated part, or with adjacent pairs) two neighbouring vectors
  const int n_rot = a.interleaved ? 0 : a.rot / 16;   // vector pairs (v, v + n_rot)
  const int v0 = j < n_rot ? j : 2 * j, v1 = j < n_rot ? j + n_rot : 2 * j + 1;
  const bool turns = !is_v && (a.interleaved ? 16 * j < a.rot : j < n_rot);   // rot is a multiple of 16

  const long long stride = is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride);
  const __nv_bfloat16* src = (is_q ? a.q : (is_v ? a.v : a.k)) + tok0 * stride + g * D;
  grid_dependency_wait();              // launched while the kernel before ends
  uint4 u0[kTokens], u1[kTokens];
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    const __nv_bfloat16* at = src + min(n, n_tok - 1) * stride;
    u0[n] = *reinterpret_cast<const uint4*>(at + 8 * v0);
    u1[n] = *reinterpret_cast<const uint4*>(at + 8 * v1);
  }
  const __nv_bfloat16* weight = is_q ? a.q_weight : (is_v ? nullptr : a.k_weight);
  F2 w0[4], w1[4];
  if (weight) {
    unpack8(*reinterpret_cast<const uint4*>(weight + 8 * v0), w0);
    unpack8(*reinterpret_cast<const uint4*>(weight + 8 * v1), w1);
  }
  const bool any_weight = __any_sync(0xffffffffu, weight != nullptr);
  float scale = 0.f;
  bool scale_ok = true;
  if (FP8 && !is_q) {
    const float ks = __ldg(a.k_scale + g), vs = __ldg(a.v_scale + g);
    scale_ok = ks > 0.f && ks <= 3.402823466e38f && vs > 0.f && vs <= 3.402823466e38f;
    scale = is_v ? vs : ks;
  }

  // token n's row of the angle table, or -1 outside it; CACHED: its row of the [rows, Hkv, D]
  // view of the cache, as kv_append places it, or -1 (outside the table, too: the cache keeps
  // what it holds)
  auto find = [&](int n, long long& angle_row, long long& dst) {
    const int tok = tok0 + n, b = tok / a.T;
    const long long pos = (a.pos0 ? (long long)__ldg(a.pos0 + b) : 0) + (tok - b * a.T);
    angle_row = a.rot == 0 ? 0 : (pos >= 0 && pos < a.rope_rows ? pos : -1);
    dst = -1;
    if (!CACHED || angle_row < 0) return;
    if (pos < 0 || pos >= (a.page_table ? (long long)a.max_blocks * kPageTokens : (long long)a.capacity)) {
      atomicOr(a.status, DEV_APPEND_RANGE);
    } else if (!a.page_table) {
      dst = (long long)b * a.capacity + pos;
    } else {
      const int blk = __ldg(a.page_table + (long long)b * a.max_blocks + pos / kPageTokens);
      if (blk >= 0 && blk < a.num_blocks) dst = (long long)blk * kPageTokens + pos % kPageTokens;
      else atomicOr(a.status, DEV_PAGE_ID);
    }
  };
  long long own_row = 0, own_dst = -1;   // kTokens == 1: each thread looks for itself
  if constexpr (kTokens == 1) {
    find(0, own_row, own_dst);
    if (own_row < 0 && j == 0) atomicOr(a.status, DEV_POSITION);
  } else {
    constexpr int kSide = 8;             // threads per token
    for (int i = threadIdx.x; i < n_tok * kSide; i += blockDim.x) {
      const int n = i / kSide, part = i % kSide;
      long long at, dst;
      find(n, at, dst);
      if (at >= 0)
        for (int e = 4 * part; e < a.rot; e += 4 * kSide)
          *reinterpret_cast<float4*>(&angles[n][e]) = __ldg(reinterpret_cast<const float4*>(a.rope + at * a.rot + e));
      if (part == 0) {
        in_table[n] = at >= 0;
        if (at < 0) atomicOr(a.status, DEV_POSITION);
        cache_row[n] = dst;
      }
    }
    __syncthreads();
  }

  // dense rows (q_out, k_out) step from token to token
  const bool dense = is_q || !CACHED;
  const int heads = is_q ? a.Hq : a.Hkv;
  __nv_bfloat16* out = (is_q ? a.q_out : a.k_out) + ((long long)tok0 * heads + g) * D;

#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    if (kTokens > 1 && n >= n_tok) break;
    const bool pos_ok = kTokens == 1 ? own_row >= 0 : in_table[n] != 0;
    const long long dst_row = kTokens == 1 ? own_dst : cache_row[n];
    F2 x0[4], x1[4];
    unpack8(u0[n], x0);
    unpack8(u1[n], x1);
    if (any_weight) {
      F2 sq = mul2(x0[0], x0[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) sq = fma2(x0[i], x0[i], sq);
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = fma2(x1[i], x1[i], sq);
      float ss = parts(sq).x + parts(sq).y;
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (weight) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        const F2 rr = f2(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x0[i] = mul2(x0[i], mul2(w0[i], rr));
          x1[i] = mul2(x1[i], mul2(w1[i], rr));
        }
      }
    }
    if (turns && pos_ok) {
      F2 c[4], s[4];
      const float* angle = kTokens == 1 ? a.rope + own_row * a.rot : angles[n];
      load8f(angle + 8 * j, c);
      load8f(angle + a.rot / 2 + 8 * j, s);
      if (!a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 p = x0[i], q = x1[i];
          x0[i] = fma2(neg2(q), s[i], mul2(p, c[i]));
          x1[i] = fma2(p, s[i], mul2(q, c[i]));
        }
      } else {
        auto turn = [](F2 x, float c, float s) {
          const float2 v = parts(x);
          return f2(v.x * c - v.y * s, v.y * c + v.x * s);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 ca = parts(c[i / 2]), sa = parts(s[i / 2]), cb = parts(c[2 + i / 2]), sb = parts(s[2 + i / 2]);
          x0[i] = turn(x0[i], i & 1 ? ca.y : ca.x, i & 1 ? sa.y : sa.x);
          x1[i] = turn(x1[i], i & 1 ? cb.y : cb.x, i & 1 ? sb.y : sb.x);
        }
      }
    }
    if (!live) continue;
    if (dense) {
      if (!pos_ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x0[i] = x1[i] = f2(NAN, NAN);
      }
      __nv_bfloat16* dst = out + (long long)n * heads * D;
      store8(dst + 8 * v0, x0);
      store8(dst + 8 * v1, x1);
      continue;
    }
    if (dst_row < 0) continue;
    const long long at = (dst_row * a.Hkv + g) * D;
    void* cache = is_v ? a.v_cache : a.k_cache;
    if constexpr (FP8) {
      if (!scale_ok) {
        if (j == 0) atomicOr(a.status, DEV_SCALE);
        continue;
      }
      uint8_t* dst = static_cast<uint8_t*>(cache) + at;
      store8_e4m3(dst + 8 * v0, x0, scale);
      store8_e4m3(dst + 8 * v1, x1, scale);
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + at;
      if (is_v) {   // as it came
        *reinterpret_cast<uint4*>(dst + 8 * v0) = u0[n];
        *reinterpret_cast<uint4*>(dst + 8 * v1) = u1[n];
      } else {
        store8(dst + 8 * v0, x0);
        store8(dst + 8 * v1, x1);
      }
    }
  }
}

// One thread per (position, pair): the angle position * theta^(-2 i / rot) in 64 bits,
// where a far position's angle keeps its fraction (in fp32 a position of 2^20 already
// costs 2^-4 radians), its cosine and sine rounded to fp32.
__global__ void __launch_bounds__(256) rope_table_kernel(float* table, int rows, int rot, double theta) {
  const int half = rot / 2;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)rows * half) return;
  const long long pos = i / half;
  const int k = (int)(i - pos * half);
  double s, c;
  sincos((double)pos * pow(theta, -2.0 * k / rot), &s, &c);
  table[pos * rot + k] = (float)c;
  table[pos * rot + half + k] = (float)s;
}

}  // namespace

namespace {
// Warps of a launch at one token each from which two, and four, tokens per warp pay.  Measured
// (us at 1, 2, 4 tokens per warp): 19200 warps 10.8, 9.6, 11.5; 38400 19.9, 17.3, 17.0; 196608
// 110, 92, 80; 192 (a decode step) 3.5, 4.9.
constexpr long long kTwoFrom = 9600, kFourFrom = 32000;

template <int D, int kTokens, bool CACHED, bool FP8>
cudaError_t run_norm_rope(const NormRopeLaunch& a, int head_groups, cudaStream_t stream) {
  const long long token_groups = ((long long)a.B * a.T + kTokens - 1) / kTokens;
  // warps per CTA: the head groups in the fewest CTAs of at most eight, evenly
  const int head_blocks = (head_groups + 7) / 8, warps = (head_groups + head_blocks - 1) / head_blocks;
  if (token_groups * head_blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_beside(norm_rope_kernel<D, kTokens, CACHED, FP8>, dim3((unsigned)(token_groups * head_blocks)),
                       32 * warps, 0, stream, a, head_blocks);
}

template <int D, bool CACHED, bool FP8>
cudaError_t run_norm_rope(const NormRopeLaunch& a, cudaStream_t stream) {
  const int heads = 32 / (D / 16), groups = (a.Hq + a.Hkv * (CACHED ? 2 : 1) + heads - 1) / heads;
  const long long warps = (long long)a.B * a.T * groups;
  if (warps >= kFourFrom) return run_norm_rope<D, 4, CACHED, FP8>(a, groups, stream);
  return warps >= kTwoFrom ? run_norm_rope<D, 2, CACHED, FP8>(a, groups, stream)
                           : run_norm_rope<D, 1, CACHED, FP8>(a, groups, stream);
}

template <int D>
cudaError_t run_norm_rope(const NormRopeLaunch& a, cudaStream_t stream) {
  if (!a.cached) return run_norm_rope<D, false, false>(a, stream);
  return a.fp8 ? run_norm_rope<D, true, true>(a, stream) : run_norm_rope<D, true, false>(a, stream);
}
}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t stream) {
  return a.d == 128 ? run_norm_rope<128>(a, stream) : run_norm_rope<64>(a, stream);
}

cudaError_t launch_rope_table(float* table, int rows, int rot, double theta, cudaStream_t stream) {
  const long long n = (long long)rows * (rot / 2);
  const long long blocks = (n + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  rope_table_kernel<<<(unsigned)blocks, 256, 0, stream>>>(table, rows, rot, theta);
  return cudaGetLastError();
}

}  // namespace kvattn
