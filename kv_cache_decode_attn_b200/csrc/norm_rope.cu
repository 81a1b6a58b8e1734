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
// shuffles).
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace kvattn {
namespace {

__device__ __forceinline__ void load8(const __nv_bfloat16* src, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(src);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// codes of x / s, each quotient one IEEE division
__device__ __forceinline__ void store8_e4m3(uint8_t* dst, const float (&x)[8], float s) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
  *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D>
__global__ void __launch_bounds__(256) norm_rope_kernel(const NormRopeLaunch a) {
  constexpr int kLanes = D / 16;   // threads per row
  const int rows_per_token = a.Hq + a.Hkv * (a.cached ? 2 : 1);   // q heads, K heads, V heads
  const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  const int j = threadIdx.x % kLanes;
  const long long n_rows = (long long)a.B * a.T * rows_per_token;
  const bool live = row < n_rows;
  const long long tok = live ? row / rows_per_token : 0;
  const int h = live ? (int)(row - tok * rows_per_token) : 0;
  const int b = (int)(tok / a.T), t = (int)(tok - (long long)b * a.T);
  const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
  const int g = is_q ? 0 : (is_v ? h - a.Hq - a.Hkv : h - a.Hq);   // KV head

  // this thread's two vectors of 8 values: both halves of its rotated pairs, or (past the
  // rotated part, or with adjacent pairs) two neighbouring vectors
  const int n_rot = a.interleaved ? 0 : a.rot / 16;   // vector pairs (v, v + n_rot)
  const int v0 = j < n_rot ? j : 2 * j, v1 = j < n_rot ? j + n_rot : 2 * j + 1;

  const __nv_bfloat16* src = is_q   ? a.q + tok * a.q_stride + (long long)h * D
                             : is_v ? a.v + tok * a.v_stride + (long long)g * D
                                    : a.k + tok * a.k_stride + (long long)g * D;
  float x0[8], x1[8];
  load8(src + 8 * v0, x0);
  load8(src + 8 * v1, x1);
  const long long pos = (a.pos0 ? (long long)__ldg(a.pos0 + b) : 0) + t;
  const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.rope_rows);

  const __nv_bfloat16* w = is_q ? a.q_weight : (is_v ? nullptr : a.k_weight);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if (!live) return;
  if (w) {
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
    float w0[8], w1[8];
    load8(w + 8 * v0, w0);
    load8(w + 8 * v1, w1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x0[i] *= r * w0[i];
      x1[i] *= r * w1[i];
    }
  }
  if (!is_v && pos_ok && a.rot > 0) {
    const float* tab = a.rope + pos * a.rot;
    if (!a.interleaved) {
      if (j < n_rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float c = __ldg(tab + 8 * j + i), s = __ldg(tab + a.rot / 2 + 8 * j + i);
          const float p = x0[i], q = x1[i];
          x0[i] = p * c - q * s;
          x1[i] = q * c + p * s;
        }
      }
    } else {
      auto turn = [&](float (&x)[8], int v) {
        if (8 * v >= a.rot) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = __ldg(tab + 4 * v + i), s = __ldg(tab + a.rot / 2 + 4 * v + i);
          const float p = x[2 * i], q = x[2 * i + 1];
          x[2 * i] = p * c - q * s;
          x[2 * i + 1] = q * c + p * s;
        }
      };
      turn(x0, v0);
      turn(x1, v1);
    }
  }
  if (!pos_ok) {
    if (j == 0) atomicOr(a.status, DEV_POSITION);
    if (!is_q && a.cached) return;   // the cache keeps what it holds
#pragma unroll
    for (int i = 0; i < 8; ++i) x0[i] = x1[i] = NAN;
  }
  if (is_q || !a.cached) {
    __nv_bfloat16* dst = is_q ? a.q_out + (tok * a.Hq + h) * D : a.k_out + (tok * a.Hkv + g) * D;
    store8(dst + 8 * v0, x0);
    store8(dst + 8 * v1, x1);
    return;
  }
  // K or V: the token's row of the cache, as kv_append places it
  long long dst_row;
  if (!a.page_table) {
    if (pos < 0 || pos >= a.capacity) {
      if (j == 0) atomicOr(a.status, DEV_APPEND_RANGE);
      return;
    }
    dst_row = ((long long)b * a.capacity + pos) * a.Hkv + g;
  } else {
    const long long blk_idx = pos / kPageTokens;
    if (pos < 0 || blk_idx >= a.max_blocks) {
      if (j == 0) atomicOr(a.status, DEV_APPEND_RANGE);
      return;
    }
    const int blk = __ldg(a.page_table + (long long)b * a.max_blocks + blk_idx);
    if (blk < 0 || blk >= a.num_blocks) {
      if (j == 0) atomicOr(a.status, DEV_PAGE_ID);
      return;
    }
    dst_row = ((long long)blk * kPageTokens + pos % kPageTokens) * a.Hkv + g;
  }
  void* cache = is_v ? a.v_cache : a.k_cache;
  if (a.fp8) {
    const float sk = __ldg(a.k_scale + g), sv = __ldg(a.v_scale + g);
    if (!(sk > 0.f && sk <= 3.402823466e38f && sv > 0.f && sv <= 3.402823466e38f)) {
      if (j == 0) atomicOr(a.status, DEV_SCALE);
      return;
    }
    uint8_t* dst = static_cast<uint8_t*>(cache) + dst_row * D;
    store8_e4m3(dst + 8 * v0, x0, is_v ? sv : sk);
    store8_e4m3(dst + 8 * v1, x1, is_v ? sv : sk);
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + dst_row * D;
    store8(dst + 8 * v0, x0);
    store8(dst + 8 * v1, x1);
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

cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t stream) {
  const long long rows = (long long)a.B * a.T * (a.Hq + a.Hkv * (a.cached ? 2 : 1));
  const int per_block = 256 / (a.d / 16);
  const long long blocks = (rows + per_block - 1) / per_block;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (a.d == 128) norm_rope_kernel<128><<<(unsigned)blocks, 256, 0, stream>>>(a);
  else norm_rope_kernel<64><<<(unsigned)blocks, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rope_table(float* table, int rows, int rot, double theta, cudaStream_t stream) {
  const long long n = (long long)rows * (rot / 2);
  const long long blocks = (n + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  rope_table_kernel<<<(unsigned)blocks, 256, 0, stream>>>(table, rows, rot, theta);
  return cudaGetLastError();
}

}  // namespace kvattn
