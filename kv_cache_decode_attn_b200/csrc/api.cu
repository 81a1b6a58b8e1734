// C ABI of the attention library: argument checks, workspace layout, tensor-map
// encoding and kernel dispatch.  The declarations and their contracts are in
// include/attn.h.  Nothing here allocates device memory.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <mutex>

#include "../../include/attn.h"
#include "internal.h"

namespace kvattn {

// Sticky device status word (ATTN_DEV_* bits), one per device that loads the library.
__device__ unsigned g_status_word;

namespace {

constexpr int kMaxDevices = 64;

unsigned* status_ptr() {
  static unsigned* ptrs[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
    ptrs[dev] = static_cast<unsigned*>(p);
  }
  return ptrs[dev];
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

int encode_tmap_nd(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                   const cuuint64_t* strides_bytes, const cuuint32_t* box, int elem_bytes) {
  auto fn = get_encode_fn();
  if (!fn || rank < 1 || rank > 5 || (elem_bytes != 1 && elem_bytes != 2)) return 1;
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUtensorMapDataType dt = elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto encode = [&] {
    return fn(map, dt, (cuuint32_t)rank, const_cast<void*>(base), dims, strides_bytes, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return 0;
  // this driver call wants the device's context on the calling thread, which a host thread has
  // only from its first runtime call that needs one
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode() ? 0 : 1;
}

int encode_tmap_3d(CUtensorMap* map, const void* base, uint64_t dim0, uint64_t dim1, uint64_t dim2,
                   uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0, uint32_t box1, uint32_t box2,
                   int elem_bytes) {
  cuuint64_t dims[3] = {dim0, dim1, dim2};
  cuuint64_t strides[2] = {stride1_bytes, stride2_bytes};
  cuuint32_t box[3] = {box0, box1, box2};
  return encode_tmap_nd(map, base, 3, dims, strides, box, elem_bytes);
}

}  // namespace kvattn

using namespace kvattn;

namespace {

// Longest selected range of a windowed decode: the first tokens' blocks, and the keys
// from the first query's window on, rounded down to a whole block.
int window_max_keys(int max_seqlen_k, int T, int window, int sinks) {
  const long long s16 = ((long long)sinks + kPageTokens - 1) / kPageTokens * kPageTokens;
  return (int)std::min<long long>(max_seqlen_k, s16 + window + T - 1 + kPageTokens - 1);
}

struct DecodeLayout {
  int R, chunk, max_chunks;
  int balanced, n_chunks;   // balanced split: chunks over the batch (per KV head)
  int stream;               // CTAs per KV head with even shares of its tiles
  int direct;               // one chunk per sequence, no combine
  size_t o_bytes, lse_offset, plan_offset, total;
};

// sel: the windowed and shared-prefix calls' splitting, max_seqlen_k being the longest selected range;
// whole: outputs may come from one CTA per (sequence, KV head)
bool decode_layout(int B, int T, int Hq, int Hkv, int d, int max_seqlen_k, int num_splits, bool fp8,
                   DecodeLayout* out, bool sel = false, bool whole = false) {
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || max_seqlen_k < 1 || num_splits < 0) return false;
  if (max_seqlen_k > kMaxDecodeSeqlen) return false;
  if (d != 64 && d != 128) return false;
  DecodeLayout L;
  L.R = (Hq / Hkv) * T;
  L.chunk = decode_chunk_tokens(B, T, Hq / Hkv, Hkv, max_seqlen_k, num_splits, fp8);
  L.max_chunks = (int)(((long long)max_seqlen_k + L.chunk - 1) / L.chunk);
  L.balanced = decode_balanced(B, T, Hq / Hkv, num_splits, fp8) ? 1 : 0;
  L.n_chunks = 0;
  size_t items = (size_t)B * Hkv * L.max_chunks;
  L.stream = 0;
  const bool tc = decode_uses_tc(L.R, fp8);
  L.direct = whole && num_splits == 0 &&
             decode_direct((long long)B * Hkv * (tc ? decode_row_tiles(T, Hq / Hkv) : 1), max_seqlen_k, tc);
  if (L.direct) {
    L.chunk = (max_seqlen_k + kDecodeTile - 1) / kDecodeTile * kDecodeTile;
    L.max_chunks = 1;
    L.balanced = 0;
    items = (size_t)B * Hkv;
  } else if (sel && num_splits == 0 && !tc) {
    L.stream = decode_stream_ctas(B, L.R, Hkv, max_seqlen_k, fp8);
    if (L.stream) items = ((size_t)L.stream + B) * Hkv;
  }
  if (L.balanced) {
    // every sequence gets at least one chunk of the batch's n_chunks
    L.n_chunks = sel ? decode_balanced_chunks(B, Hkv, 1) : decode_balanced_chunks(B, Hkv);
    L.max_chunks = L.n_chunks - B + 1;   // most chunks one (sequence, KV head) can get
    items = (size_t)L.n_chunks * Hkv;
  }
  L.o_bytes = items * L.R * d * sizeof(float);
  L.lse_offset = (L.o_bytes + 255) & ~size_t(255);
  L.plan_offset = (L.lse_offset + items * L.R * sizeof(float) + 255) & ~size_t(255);
  L.total = L.plan_offset + (L.balanced ? (size_t)B * 3 * sizeof(int) : 0);
  *out = L;
  return true;
}

// With KVATTN_DEBUG set in the environment, CUDA failures are also printed to stderr.
int cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return ATTN_OK;
  static const bool debug = getenv("KVATTN_DEBUG") != nullptr;
  if (debug) fprintf(stderr, "[kvattn] %s: %s (%d)\n", where, cudaGetErrorString(e), (int)e);
  return ATTN_ERR_CUDA;
}

int prefill_impl(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse, int B, int Hq,
                 int Hkv, int N, int d, float scale, int causal, bool windowed, int window, int sinks, void* stream,
                 const char* name) {
  if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || N < 1 || Hq % Hkv) return ATTN_ERR_INVALID_ARG;
  if (o_dtype != ATTN_F32 && o_dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale) || (causal != 0 && causal != 1)) return ATTN_ERR_INVALID_ARG;
  if (windowed && (window < 1 || sinks < 0)) return ATTN_ERR_INVALID_ARG;
  if (windowed && N > kMaxDecodeSeqlen) return ATTN_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * N * Hq > INT32_MAX || (long long)B * N * Hkv > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  unsigned* st = status_ptr();
  if (!st) return ATTN_ERR_CUDA;
  PrefillLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.o_bf16 = o_dtype == ATTN_BF16;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.scale = scale;
  a.causal = causal;
  a.status = st;
  if (windowed) {   // the same keys, and no overflow
    a.window = std::min(window, N);
    a.sinks = std::min(sinks, N);
  }
  return cuda_status(launch_prefill(a, static_cast<cudaStream_t>(stream)), name);
}

}  // namespace

extern "C" {

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported configuration";
    case ATTN_ERR_WORKSPACE: return "workspace missing or too small";
    case ATTN_ERR_CUDA: return "CUDA error";
    case ATTN_ERR_DEVICE: return "device-side error flagged";
    case ATTN_ERR_NO_BLOCKS: return "block pool exhausted";
    default: return "unknown status";
  }
}

int64_t kv_cache_bytes(int n_layers, int batch, int64_t tokens, int n_kv_heads, int head_dim, int elem_bytes) {
  if (n_layers <= 0 || batch <= 0 || tokens <= 0 || n_kv_heads <= 0 || head_dim <= 0 || elem_bytes <= 0) return -1;
  const int64_t factors[6] = {n_layers, batch, tokens, n_kv_heads, head_dim, elem_bytes};
  int64_t r = 2;
  for (int i = 0; i < 6; ++i) {
    if (r > INT64_MAX / factors[i]) return -1;
    r *= factors[i];
  }
  return r;
}

int attn_get_device_status(int clear) {
  unsigned* p = status_ptr();
  if (!p) return ATTN_ERR_CUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return ATTN_ERR_CUDA;
  unsigned v = 0;
  if (cudaMemcpy(&v, p, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return ATTN_ERR_CUDA;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpy(p, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return ATTN_ERR_CUDA;
  }
  return (int)v;
}

size_t attn_decode_workspace_bytes(int B, int T, int Hq, int Hkv, int d, int max_seqlen_k, int num_splits) {
  // enough for attn_decode and for attn_decode_fp8 with the same arguments (their chunking differs)
  DecodeLayout L, L8;
  if (!decode_layout(B, T, Hq, Hkv, d, max_seqlen_k, num_splits, false, &L)) return 0;
  if (!decode_layout(B, T, Hq, Hkv, d, max_seqlen_k, num_splits, true, &L8)) return 0;
  return L.total > L8.total ? L.total : L8.total;
}

int attn_prefill(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse, int B, int Hq,
                 int Hkv, int N, int d, float scale, int causal, void* stream) {
  return prefill_impl(q, k, v, o, o_dtype, lse, B, Hq, Hkv, N, d, scale, causal, false, 0, 0, stream, "attn_prefill");
}

}  // extern "C"

namespace {

int decode_impl(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                bool fp8, const int32_t* seqlens_k, const int32_t* page_table, int max_blocks_per_seq,
                int num_blocks, int cache_capacity, int max_seqlen_k, void* o, int o_dtype, float* lse, int B, int T,
                int Hq, int Hkv, int d, float scale, int causal, int num_splits, void* workspace,
                size_t workspace_bytes, void* stream, const char* name, bool static_scratch = false,
                int window = 0, int sinks = 0) {
  if (!q || !k_cache || !v_cache || !seqlens_k || !o) return ATTN_ERR_INVALID_ARG;
  if (fp8 && (!k_scale || !v_scale)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_splits < 0) return ATTN_ERR_INVALID_ARG;
  if (o_dtype != ATTN_F32 && o_dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale) || (causal != 0 && causal != 1)) return ATTN_ERR_INVALID_ARG;
  const bool paged = page_table != nullptr;
  int capacity_tokens;
  if (paged) {
    if (max_blocks_per_seq < 1 || num_blocks < 1) return ATTN_ERR_INVALID_ARG;
    if ((long long)num_blocks * kPageTokens > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
    capacity_tokens = (int)std::min<long long>((long long)max_blocks_per_seq * kPageTokens, INT32_MAX);
  } else {
    if (cache_capacity < 1) return ATTN_ERR_INVALID_ARG;
    if ((long long)B * cache_capacity > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
    capacity_tokens = cache_capacity;
  }
  if (max_seqlen_k == 0) max_seqlen_k = std::min(capacity_tokens, kMaxDecodeSeqlen);
  if (max_seqlen_k < T || max_seqlen_k > capacity_tokens) return ATTN_ERR_INVALID_ARG;
  if (max_seqlen_k > kMaxDecodeSeqlen) return ATTN_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (Hq / Hkv > 128) return ATTN_ERR_UNSUPPORTED;                       // one token's heads must fit a row tile
  if (fp8 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if (window >= max_seqlen_k || sinks >= max_seqlen_k) window = 0;   // every key up to the own one: plain decode
  const int max_keys = window > 0 ? window_max_keys(max_seqlen_k, T, window, sinks) : max_seqlen_k;
  DecodeLayout L;
  if (!decode_layout(B, T, Hq, Hkv, d, max_keys, num_splits, fp8, &L, window > 0, window > 0)) return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < L.total) return ATTN_ERR_WORKSPACE;
  if (static_scratch) {
    // attn_decode_noalloc: the library's own array, looked up only once the request is known to be valid
    workspace = noalloc_scratch();
    if (!workspace) return ATTN_ERR_CUDA;
  }
  if (!workspace || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
  unsigned* st = status_ptr();
  if (!st) return ATTN_ERR_CUDA;
  if (!fp8 && num_splits == 0 && T >= kDecodeViaPrefillT && (long long)B * T * Hq <= INT32_MAX) {
    // a prompt chunk against a cached prefix: the prefill kernel's cached form computes the
    // same rows (bottom-right causal alignment, the same length rules with max_seqlen_k) faster;
    // the workspace goes unused
    PrefillLaunch pa;
    pa.q = q;
    pa.k = k_cache;
    pa.v = v_cache;
    pa.o = o;
    pa.o_bf16 = o_dtype == ATTN_BF16;
    pa.lse = lse;
    pa.B = B;
    pa.Hq = Hq;
    pa.Hkv = Hkv;
    pa.N = T;
    pa.d = d;
    pa.scale = scale;
    pa.causal = causal;
    pa.status = st;
    pa.seqlens = seqlens_k;
    pa.page_table = page_table;
    pa.capacity = cache_capacity;
    pa.max_blocks = max_blocks_per_seq;
    pa.num_blocks = num_blocks;
    pa.max_seqlen = max_seqlen_k;
    pa.window = window;
    pa.sinks = sinks;
    return cuda_status(launch_prefill(pa, static_cast<cudaStream_t>(stream)), name);
  }
  DecodeLaunch a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.seqlens = seqlens_k;
  a.page_table = page_table;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.capacity = cache_capacity;
  a.max_seqlen = max_seqlen_k;
  a.o = o;
  a.o_bf16 = o_dtype == ATTN_BF16;
  a.lse = lse;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.scale = scale;
  a.causal = causal;
  a.chunk = L.chunk;
  a.max_chunks = L.max_chunks;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.lse_offset);
  a.balanced = L.balanced;
  a.n_chunks = L.n_chunks;
  a.plan = L.balanced ? reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + L.plan_offset) : nullptr;
  a.status = st;
  a.fp8 = fp8 ? 1 : 0;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  if (window > 0) {
    a.sel.select = 1;
    a.sel.window = window;
    a.sel.sinks = sinks;
    a.stream = L.stream;
    a.direct = L.direct;
  }
  return cuda_status(launch_decode(a, static_cast<cudaStream_t>(stream)), name);
}

// Shared-prefix decode: the launches' parts of the workspace.  The prefix's partials are
// those of one sequence with B * T query tokens; the own part's follow.
struct SharedLayout {
  int together;   // as if nothing were shared: own is the layout of the whole
  int pre_chunk, pre_chunks, pre_stream;
  size_t pre_lse_offset, own_offset, total;
  DecodeLayout own;
};

bool shared_layout(int B, int T, int Hq, int Hkv, int d, int max_seqlen_k, int prefix_blocks, int num_splits, bool fp8,
                   SharedLayout* out) {
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_splits < 0 || prefix_blocks < 1) return false;
  if (max_seqlen_k < 1 || max_seqlen_k > kMaxDecodeSeqlen || prefix_blocks > kMaxDecodeSeqlen / kPageTokens) return false;
  if ((long long)B * T > INT32_MAX / 128 || Hq / Hkv > 128) return false;
  const int P = prefix_blocks * kPageTokens;
  if (max_seqlen_k - P < T) return false;
  SharedLayout s = {};
  if (num_splits == 0 && decode_shared_together(B, T, Hq / Hkv, Hkv, max_seqlen_k, P, fp8)) {
    s.together = 1;
    if (!decode_layout(B, T, Hq, Hkv, d, max_seqlen_k, 0, fp8, &s.own, true, true)) return false;
    s.total = s.own.total;
    *out = s;
    return true;
  }
  if (!decode_layout(B, T, Hq, Hkv, d, max_seqlen_k - P, num_splits, fp8, &s.own, true)) return false;
  const int R = B * T * (Hq / Hkv);   // the prefix's query rows per KV head
  s.pre_chunk = prefix_chunk_tokens(B * T, Hq / Hkv, Hkv, P, num_splits, fp8);
  s.pre_chunks = (P + s.pre_chunk - 1) / s.pre_chunk;
  s.pre_stream = num_splits == 0 && !decode_uses_tc(R, fp8) ? decode_stream_ctas(1, R, Hkv, P, fp8) : 0;
  const size_t rows = (s.pre_stream ? s.pre_stream + 1 : s.pre_chunks) * (size_t)Hkv * R;
  s.pre_lse_offset = (rows * d * sizeof(float) + 255) & ~size_t(255);
  s.own_offset = (s.pre_lse_offset + rows * sizeof(float) + 255) & ~size_t(255);
  s.total = s.own_offset + s.own.total;
  *out = s;
  return true;
}

int shared_impl(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                bool fp8, const int32_t* seqlens_k, const int32_t* page_table, int max_blocks_per_seq, int num_blocks,
                const int32_t* prefix_table, int prefix_blocks, int max_seqlen_k, void* o, int o_dtype, float* lse,
                int B, int T, int Hq, int Hkv, int d, float scale, int causal, int num_splits, void* workspace,
                size_t workspace_bytes, void* stream, const char* name) {
  if (!q || !k_cache || !v_cache || !seqlens_k || !page_table || !o) return ATTN_ERR_INVALID_ARG;
  if (fp8 && (!k_scale || !v_scale)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_splits < 0) return ATTN_ERR_INVALID_ARG;
  if (o_dtype != ATTN_F32 && o_dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale) || (causal != 0 && causal != 1)) return ATTN_ERR_INVALID_ARG;
  if (max_blocks_per_seq < 1 || num_blocks < 1 || prefix_blocks < 0 || prefix_blocks > max_blocks_per_seq)
    return ATTN_ERR_INVALID_ARG;
  if (prefix_blocks == 0)   // nothing shared: plain decode, with the same splitting and workspace rules
    return decode_impl(q, k_cache, v_cache, k_scale, v_scale, fp8, seqlens_k, page_table, max_blocks_per_seq,
                       num_blocks, 0, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, causal, num_splits,
                       workspace, workspace_bytes, stream, name);
  if (!prefix_table) return ATTN_ERR_INVALID_ARG;
  if ((long long)num_blocks * kPageTokens > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  const int capacity = (int)std::min<long long>((long long)max_blocks_per_seq * kPageTokens, INT32_MAX);
  if (max_seqlen_k == 0) max_seqlen_k = std::min(capacity, kMaxDecodeSeqlen);
  if (max_seqlen_k < 0 || max_seqlen_k > capacity) return ATTN_ERR_INVALID_ARG;
  if (max_seqlen_k > kMaxDecodeSeqlen) return ATTN_ERR_UNSUPPORTED;
  // every sequence holds the whole prefix and its T new tokens
  if ((long long)prefix_blocks * kPageTokens + T > max_seqlen_k) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (Hq / Hkv > 128 || (fp8 && d != 128)) return ATTN_ERR_UNSUPPORTED;
  if ((long long)B * T > INT32_MAX / 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  SharedLayout s;
  if (!shared_layout(B, T, Hq, Hkv, d, max_seqlen_k, prefix_blocks, num_splits, fp8, &s)) return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < s.total || !workspace || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
  unsigned* st = status_ptr();
  if (!st) return ATTN_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  // the prefix: one sequence whose queries are the whole batch's, every key visible to all
  DecodeLaunch pre = {};
  pre.q = q;
  pre.k = k_cache;
  pre.v = v_cache;
  pre.page_table = prefix_table;
  pre.max_blocks = prefix_blocks;
  pre.num_blocks = num_blocks;
  pre.max_seqlen = prefix_blocks * kPageTokens;
  pre.B = 1;
  pre.T = B * T;
  pre.Hq = Hq;
  pre.Hkv = Hkv;
  pre.d = d;
  pre.scale = scale;
  pre.chunk = s.pre_chunk;
  pre.max_chunks = s.pre_chunks;
  pre.part_o = reinterpret_cast<float*>(ws);
  pre.part_lse = reinterpret_cast<float*>(ws + s.pre_lse_offset);
  pre.status = st;
  pre.fp8 = fp8 ? 1 : 0;
  pre.k_scale = k_scale;
  pre.v_scale = v_scale;
  pre.sel.select = 1;
  pre.sel.fixed_len = prefix_blocks * kPageTokens;
  pre.stream = s.pre_stream;
  pre.early = 1;
  // each sequence's own keys, and the merge of both parts
  DecodeLaunch own = pre;
  own.seqlens = seqlens_k;
  own.page_table = page_table;
  own.max_blocks = max_blocks_per_seq;
  own.max_seqlen = max_seqlen_k;
  own.o = o;
  own.o_bf16 = o_dtype == ATTN_BF16;
  own.lse = lse;
  own.B = B;
  own.T = T;
  own.causal = causal;
  own.chunk = s.own.chunk;
  own.max_chunks = s.own.max_chunks;
  own.part_o = reinterpret_cast<float*>(ws + s.own_offset);
  own.part_lse = reinterpret_cast<float*>(ws + s.own_offset + s.own.lse_offset);
  own.balanced = s.own.balanced;
  own.n_chunks = s.own.n_chunks;
  own.plan = s.own.balanced ? reinterpret_cast<int*>(ws + s.own_offset + s.own.plan_offset) : nullptr;
  own.stream = s.own.stream;
  own.early = 0;
  own.fence = 1;
  own.sel.fixed_len = 0;
  own.sel.min_len = prefix_blocks * kPageTokens + T;
  if (s.together) {
    own.direct = s.own.direct;
    own.early = own.fence = 0;
    own.sel.prefix = prefix_table;
    own.sel.prefix_blocks = prefix_blocks;
    return cuda_status(launch_decode(own, static_cast<cudaStream_t>(stream)), name);
  }
  own.sel.skip = prefix_blocks * kPageTokens;
  own.pre_o = pre.part_o;
  own.pre_lse = pre.part_lse;
  own.pre_chunks = s.pre_chunks;
  own.pre_stream = s.pre_stream;
  own.pre_tiles = prefix_blocks * kPageTokens / kDecodeTile + (prefix_blocks * kPageTokens % kDecodeTile != 0);
  // The prefix goes first, one wave of CTAs; the own part's CTAs may start at once and take the
  // SMs as the prefix's leave them, its launch ends after the prefix's, and the combine waits for
  // both.  One CTA of each per SM, side by side, measured no better: 102 us against 95 for 64
  // sequences of about 1000 own keys behind 32K, 31 against 33 for short ones behind 4K.
  cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_decode_split(pre, st_);
  if (e == cudaSuccess) e = launch_decode_split(own, st_);
  if (e == cudaSuccess) e = launch_decode_combine(own, st_);
  return cuda_status(e, name);
}

int prefill_cache_impl(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens_k,
                       const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity, void* o,
                       int o_dtype, float* lse, int B, int Nq, int Hq, int Hkv, int d, float scale, int causal,
                       bool windowed, int window, int sinks, void* stream, const char* name) {
  if (!q || !k_cache || !v_cache || !seqlens_k || !o) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Nq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv) return ATTN_ERR_INVALID_ARG;
  if (o_dtype != ATTN_F32 && o_dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale) || (causal != 0 && causal != 1)) return ATTN_ERR_INVALID_ARG;
  if (page_table) {
    if (max_blocks_per_seq < 1 || num_blocks < 1) return ATTN_ERR_INVALID_ARG;
    if ((long long)num_blocks * kPageTokens > INT32_MAX || (long long)max_blocks_per_seq * kPageTokens > INT32_MAX)
      return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_blocks_per_seq * kPageTokens < Nq) return ATTN_ERR_INVALID_ARG;
  } else {
    if (cache_capacity < Nq) return ATTN_ERR_INVALID_ARG;
  }
  if (windowed && (window < 1 || sinks < 0)) return ATTN_ERR_INVALID_ARG;
  const int max_keys = page_table ? max_blocks_per_seq * kPageTokens : cache_capacity;
  if (windowed && max_keys > kMaxDecodeSeqlen) return ATTN_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Nq * Hq > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  unsigned* st = status_ptr();
  if (!st) return ATTN_ERR_CUDA;
  PrefillLaunch a;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.o = o;
  a.o_bf16 = o_dtype == ATTN_BF16;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = Nq;
  a.d = d;
  a.scale = scale;
  a.causal = causal;
  a.status = st;
  a.seqlens = seqlens_k;
  a.page_table = page_table;
  a.capacity = cache_capacity;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  if (windowed) {   // the same keys, and no overflow
    a.window = std::min(window, max_keys);
    a.sinks = std::min(sinks, max_keys);
  }
  return cuda_status(launch_prefill(a, static_cast<cudaStream_t>(stream)), name);
}

// Whether n1 bytes at p1 and n2 bytes at p2 share any.
bool overlap(const void* p1, size_t n1, const void* p2, size_t n2) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p1), b = reinterpret_cast<uintptr_t>(p2);
  return a < b + n2 && b < a + n1;
}

// The checks qk_norm_rope and kv_append_norm_rope share; fills the launch's common part.
int norm_rope_args(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                   void* q_out, void* k_out, const void* q_weight, const void* k_weight, float eps, const float* rope,
                   int rope_rows, int rot_dim, int interleaved, const int32_t* pos0, int B, int T, int Hq, int Hkv,
                   int d, bool cached, NormRopeLaunch* out) {
  if (!q || !k || !q_out || (cached ? !v : !k_out)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || rot_dim < 0 || (interleaved != 0 && interleaved != 1))
    return ATTN_ERR_INVALID_ARG;
  if ((rot_dim > 0) != (rope != nullptr) || (rot_dim > 0 && rope_rows < 1)) return ATTN_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && (!(eps > 0.f) || !isfinite(eps))) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (rot_dim > d) return ATTN_ERR_INVALID_ARG;
  if (rot_dim % 16) return ATTN_ERR_UNSUPPORTED;
  if ((long long)B * T > INT32_MAX || (long long)Hq + 2LL * Hkv > INT32_MAX / 128) return ATTN_ERR_UNSUPPORTED;
  if (q_stride < (int64_t)Hq * d || k_stride < (int64_t)Hkv * d || (cached && v_stride < (int64_t)Hkv * d) ||
      q_stride % 8 || k_stride % 8 || (cached && v_stride % 8))
    return ATTN_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * T;
  if (q_stride > INT64_MAX / 4 / n || k_stride > INT64_MAX / 4 / n || (cached && v_stride > INT64_MAX / 4 / n))
    return ATTN_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, cached ? v : q, q_out, cached ? q_out : k_out, q_weight, k_weight, rope};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ATTN_ERR_INVALID_ARG;
  // an output may be exactly its own input; any other overlap would be read after it is written
  const size_t qn = (size_t)(n * Hq * d) * 2, kn = (size_t)(n * Hkv * d) * 2;
  auto span = [&](int64_t stride, int H) { return (size_t)((n - 1) * stride + (int64_t)H * d) * 2; };
  auto clash = [&](const void* dst, size_t bytes, const void* src, int64_t stride, int H, bool own) {
    if (own && dst == src && stride == (int64_t)H * d) return false;
    return overlap(dst, bytes, src, span(stride, H));
  };
  if (clash(q_out, qn, q, q_stride, Hq, true) || clash(q_out, qn, k, k_stride, Hkv, false)) return ATTN_ERR_INVALID_ARG;
  if (cached && clash(q_out, qn, v, v_stride, Hkv, false)) return ATTN_ERR_INVALID_ARG;
  if (!cached && (clash(k_out, kn, q, q_stride, Hq, false) || clash(k_out, kn, k, k_stride, Hkv, true) ||
                  overlap(q_out, qn, k_out, kn)))
    return ATTN_ERR_INVALID_ARG;
  NormRopeLaunch a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  a.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  a.eps = eps;
  a.rope = rope;
  a.rope_rows = rope_rows;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.pos0 = pos0;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.cached = cached ? 1 : 0;
  *out = a;
  return ATTN_OK;
}

int append_norm_rope_impl(void* k_cache, void* v_cache, const void* q, const void* k_new, const void* v_new,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride, void* q_out, const float* k_scale,
                          const float* v_scale, bool fp8, const void* q_weight, const void* k_weight, float eps,
                          const float* rope, int rope_rows, int rot_dim, int interleaved, const int32_t* cache_lens,
                          const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity, int B,
                          int T, int Hq, int Hkv, int d, void* stream, const char* name) {
  if (!k_cache || !v_cache || !cache_lens) return ATTN_ERR_INVALID_ARG;
  if (fp8 && (!k_scale || !v_scale)) return ATTN_ERR_INVALID_ARG;
  if (page_table) {
    if (max_blocks_per_seq < 1 || num_blocks < 1) return ATTN_ERR_INVALID_ARG;
  } else if (cache_capacity < 1) {
    return ATTN_ERR_INVALID_ARG;
  }
  NormRopeLaunch a;
  const int e = norm_rope_args(q, k_new, v_new, q_stride, k_stride, v_stride, q_out, nullptr, q_weight, k_weight, eps,
                               rope, rope_rows, rot_dim, interleaved, cache_lens, B, T, Hq, Hkv, d, true, &a);
  if (e != ATTN_OK) return e;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return ATTN_ERR_INVALID_ARG;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_table = page_table;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.capacity = cache_capacity;
  a.fp8 = fp8 ? 1 : 0;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  if (!(a.status = status_ptr())) return ATTN_ERR_CUDA;
  return cuda_status(launch_norm_rope(a, static_cast<cudaStream_t>(stream)), name);
}

int append_impl(void* k_cache, void* v_cache, const void* k_new, const void* v_new, const float* k_scale,
                const float* v_scale, bool fp8, const int32_t* cache_lens, const int32_t* page_table,
                int max_blocks_per_seq, int num_blocks, int cache_capacity, int B, int T, int Hkv, int d, void* stream,
                const char* name) {
  if (!k_cache || !v_cache || !k_new || !v_new || !cache_lens) return ATTN_ERR_INVALID_ARG;
  if (fp8 && (!k_scale || !v_scale)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if (page_table) {
    if (max_blocks_per_seq < 1 || num_blocks < 1) return ATTN_ERR_INVALID_ARG;
  } else if (cache_capacity < 1) {
    return ATTN_ERR_INVALID_ARG;
  }
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_new) || !aligned16(v_new))
    return ATTN_ERR_INVALID_ARG;
  unsigned* st = status_ptr();
  if (!st) return ATTN_ERR_CUDA;
  AppendLaunch a;
  a.k = k_cache;
  a.v = v_cache;
  a.k_new = k_new;
  a.v_new = v_new;
  a.cache_lens = cache_lens;
  a.page_table = page_table;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.capacity = cache_capacity;
  a.B = B;
  a.T = T;
  a.Hkv = Hkv;
  a.d = d;
  a.status = st;
  a.fp8 = fp8 ? 1 : 0;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return cuda_status(launch_append(a, static_cast<cudaStream_t>(stream)), name);
}

}  // namespace

extern "C" {

int attn_prefill_cache(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens_k,
                       const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity, void* o,
                       int o_dtype, float* lse, int B, int Nq, int Hq, int Hkv, int d, float scale, int causal,
                       void* stream) {
  return prefill_cache_impl(q, k_cache, v_cache, seqlens_k, page_table, max_blocks_per_seq, num_blocks, cache_capacity,
                            o, o_dtype, lse, B, Nq, Hq, Hkv, d, scale, causal, false, 0, 0, stream,
                            "attn_prefill_cache");
}

int attn_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens_k,
                const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity,
                int max_seqlen_k, void* o, int o_dtype, float* lse, int B, int T, int Hq, int Hkv, int d,
                float scale, int causal, int num_splits, void* workspace, size_t workspace_bytes, void* stream) {
  return decode_impl(q, k_cache, v_cache, nullptr, nullptr, false, seqlens_k, page_table, max_blocks_per_seq,
                     num_blocks, cache_capacity, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, causal,
                     num_splits, workspace, workspace_bytes, stream, "attn_decode");
}

int attn_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens_k,
                        const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity,
                        int max_seqlen_k, void* o, int o_dtype, float* lse, int B, int T, int Hq, int Hkv, int d,
                        float scale, int causal, int num_splits, void* stream) {
  return decode_impl(q, k_cache, v_cache, nullptr, nullptr, false, seqlens_k, page_table, max_blocks_per_seq,
                     num_blocks, cache_capacity, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, causal,
                     num_splits, nullptr, ATTN_DECODE_NOALLOC_SCRATCH_BYTES, stream, "attn_decode_noalloc", true);
}

int attn_decode_fp8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, const int32_t* seqlens_k, const int32_t* page_table, int max_blocks_per_seq,
                    int num_blocks, int cache_capacity, int max_seqlen_k, void* o, int o_dtype, float* lse, int B,
                    int T, int Hq, int Hkv, int d, float scale, int causal, int num_splits, void* workspace,
                    size_t workspace_bytes, void* stream) {
  return decode_impl(q, k_cache, v_cache, k_scale, v_scale, true, seqlens_k, page_table, max_blocks_per_seq,
                     num_blocks, cache_capacity, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, causal,
                     num_splits, workspace, workspace_bytes, stream, "attn_decode_fp8");
}

int attn_prefill_window(const void* q, const void* k, const void* v, void* o, int o_dtype, float* lse, int B, int Hq,
                        int Hkv, int N, int d, float scale, int window, int sinks, void* stream) {
  return prefill_impl(q, k, v, o, o_dtype, lse, B, Hq, Hkv, N, d, scale, 1, true, window, sinks, stream,
                      "attn_prefill_window");
}

int attn_prefill_cache_window(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens_k,
                              const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity,
                              void* o, int o_dtype, float* lse, int B, int Nq, int Hq, int Hkv, int d, float scale,
                              int window, int sinks, void* stream) {
  return prefill_cache_impl(q, k_cache, v_cache, seqlens_k, page_table, max_blocks_per_seq, num_blocks, cache_capacity,
                            o, o_dtype, lse, B, Nq, Hq, Hkv, d, scale, 1, true, window, sinks, stream,
                            "attn_prefill_cache_window");
}

size_t attn_decode_window_workspace_bytes(int B, int T, int Hq, int Hkv, int d, int max_seqlen_k, int window, int sinks,
                                          int num_splits) {
  if (window < 1 || sinks < 0 || T < 1 || max_seqlen_k < 1 || max_seqlen_k > kMaxDecodeSeqlen) return 0;
  if (window >= max_seqlen_k || sinks >= max_seqlen_k)
    return attn_decode_workspace_bytes(B, T, Hq, Hkv, d, max_seqlen_k, num_splits);
  const int max_keys = window_max_keys(max_seqlen_k, T, window, sinks);
  DecodeLayout L, L8;   // enough for either cache type, as attn_decode_workspace_bytes
  if (!decode_layout(B, T, Hq, Hkv, d, max_keys, num_splits, false, &L, true, true)) return 0;
  if (!decode_layout(B, T, Hq, Hkv, d, max_keys, num_splits, true, &L8, true, true)) return 0;
  return std::max(L.total, L8.total);
}

int attn_decode_window(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens_k,
                       const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity,
                       int max_seqlen_k, void* o, int o_dtype, float* lse, int B, int T, int Hq, int Hkv, int d,
                       float scale, int window, int sinks, int num_splits, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  return decode_impl(q, k_cache, v_cache, nullptr, nullptr, false, seqlens_k, page_table, max_blocks_per_seq,
                     num_blocks, cache_capacity, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, 1, num_splits,
                     workspace, workspace_bytes, stream, "attn_decode_window", false, window, sinks);
}

int attn_decode_window_fp8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int32_t* seqlens_k, const int32_t* page_table,
                           int max_blocks_per_seq, int num_blocks, int cache_capacity, int max_seqlen_k, void* o,
                           int o_dtype, float* lse, int B, int T, int Hq, int Hkv, int d, float scale, int window,
                           int sinks, int num_splits, void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  return decode_impl(q, k_cache, v_cache, k_scale, v_scale, true, seqlens_k, page_table, max_blocks_per_seq, num_blocks,
                     cache_capacity, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, 1, num_splits, workspace,
                     workspace_bytes, stream, "attn_decode_window_fp8", false, window, sinks);
}

size_t attn_decode_shared_workspace_bytes(int B, int T, int Hq, int Hkv, int d, int max_seqlen_k, int prefix_blocks,
                                          int num_splits) {
  if (prefix_blocks == 0) return attn_decode_workspace_bytes(B, T, Hq, Hkv, d, max_seqlen_k, num_splits);
  SharedLayout s, s8;   // enough for either cache type, as attn_decode_workspace_bytes
  if (!shared_layout(B, T, Hq, Hkv, d, max_seqlen_k, prefix_blocks, num_splits, false, &s)) return 0;
  if (!shared_layout(B, T, Hq, Hkv, d, max_seqlen_k, prefix_blocks, num_splits, true, &s8)) return 0;
  return std::max(s.total, s8.total);
}

int attn_decode_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* seqlens_k,
                       const int32_t* page_table, int max_blocks_per_seq, int num_blocks, const int32_t* prefix_table,
                       int prefix_blocks, int max_seqlen_k, void* o, int o_dtype, float* lse, int B, int T, int Hq,
                       int Hkv, int d, float scale, int causal, int num_splits, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return shared_impl(q, k_cache, v_cache, nullptr, nullptr, false, seqlens_k, page_table, max_blocks_per_seq, num_blocks,
                     prefix_table, prefix_blocks, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, causal,
                     num_splits, workspace, workspace_bytes, stream, "attn_decode_shared");
}

int attn_decode_shared_fp8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int32_t* seqlens_k, const int32_t* page_table,
                           int max_blocks_per_seq, int num_blocks, const int32_t* prefix_table, int prefix_blocks,
                           int max_seqlen_k, void* o, int o_dtype, float* lse, int B, int T, int Hq, int Hkv, int d,
                           float scale, int causal, int num_splits, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return shared_impl(q, k_cache, v_cache, k_scale, v_scale, true, seqlens_k, page_table, max_blocks_per_seq, num_blocks,
                     prefix_table, prefix_blocks, max_seqlen_k, o, o_dtype, lse, B, T, Hq, Hkv, d, scale, causal,
                     num_splits, workspace, workspace_bytes, stream, "attn_decode_shared_fp8");
}

int kv_append(void* k_cache, void* v_cache, const void* k_new, const void* v_new, const int32_t* cache_lens,
              const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity, int B, int T,
              int Hkv, int d, void* stream) {
  return append_impl(k_cache, v_cache, k_new, v_new, nullptr, nullptr, false, cache_lens, page_table,
                     max_blocks_per_seq, num_blocks, cache_capacity, B, T, Hkv, d, stream, "kv_append");
}

int attn_copy_blocks(void* k_pool, void* v_pool, const int32_t* src, const int32_t* dst, int n, int num_blocks,
                     int Hkv, int d, int elem_bytes, void* stream) {
  if (!k_pool || !v_pool || n < 0 || num_blocks < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if (n > 0 && (!src || !dst)) return ATTN_ERR_INVALID_ARG;
  if (n > 65535) return ATTN_ERR_UNSUPPORTED;
  if ((d != 64 && d != 128) || (elem_bytes != 1 && elem_bytes != 2)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(k_pool) || !aligned16(v_pool)) return ATTN_ERR_INVALID_ARG;
  if (n == 0) return ATTN_OK;
  const long long block_bytes = (long long)kPageTokens * Hkv * d * elem_bytes;
  if (block_bytes / 16 > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  unsigned* st = status_ptr();
  if (!st) return ATTN_ERR_CUDA;
  return cuda_status(launch_copy_blocks(k_pool, v_pool, src, dst, n, num_blocks, (int)block_bytes, st,
                                        static_cast<cudaStream_t>(stream)),
                     "attn_copy_blocks");
}

int attn_selftest_wait_timeout(void* stream) {
  unsigned* st = status_ptr();
  if (!st) return ATTN_ERR_CUDA;
  return cuda_status(launch_wait_timeout_selftest(st, static_cast<cudaStream_t>(stream)),
                     "attn_selftest_wait_timeout");
}

int kv_append_fp8(void* k_cache, void* v_cache, const void* k_new, const void* v_new, const float* k_scale,
                  const float* v_scale, const int32_t* cache_lens, const int32_t* page_table, int max_blocks_per_seq,
                  int num_blocks, int cache_capacity, int B, int T, int Hkv, int d, void* stream) {
  return append_impl(k_cache, v_cache, k_new, v_new, k_scale, v_scale, true, cache_lens, page_table,
                     max_blocks_per_seq, num_blocks, cache_capacity, B, T, Hkv, d, stream, "kv_append_fp8");
}

int qk_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, void* q_out, void* k_out,
                 const void* q_weight, const void* k_weight, float eps, const float* rope, int rope_rows, int rot_dim,
                 int interleaved, const int32_t* pos0, int B, int T, int Hq, int Hkv, int d, void* stream) {
  NormRopeLaunch a;
  const int e = norm_rope_args(q, k, nullptr, q_stride, k_stride, 0, q_out, k_out, q_weight, k_weight, eps, rope,
                               rope_rows, rot_dim, interleaved, pos0, B, T, Hq, Hkv, d, false, &a);
  if (e != ATTN_OK) return e;
  if (!(a.status = status_ptr())) return ATTN_ERR_CUDA;
  return cuda_status(launch_norm_rope(a, static_cast<cudaStream_t>(stream)), "qk_norm_rope");
}

int kv_append_norm_rope(void* k_cache, void* v_cache, const void* q, const void* k_new, const void* v_new,
                        int64_t q_stride, int64_t k_stride, int64_t v_stride, void* q_out, const void* q_weight,
                        const void* k_weight, float eps, const float* rope, int rope_rows, int rot_dim,
                        int interleaved, const int32_t* cache_lens, const int32_t* page_table, int max_blocks_per_seq,
                        int num_blocks, int cache_capacity, int B, int T, int Hq, int Hkv, int d, void* stream) {
  return append_norm_rope_impl(k_cache, v_cache, q, k_new, v_new, q_stride, k_stride, v_stride, q_out, nullptr, nullptr,
                               false, q_weight, k_weight, eps, rope, rope_rows, rot_dim, interleaved, cache_lens,
                               page_table, max_blocks_per_seq, num_blocks, cache_capacity, B, T, Hq, Hkv, d, stream,
                               "kv_append_norm_rope");
}

int kv_append_norm_rope_fp8(void* k_cache, void* v_cache, const void* q, const void* k_new, const void* v_new,
                            int64_t q_stride, int64_t k_stride, int64_t v_stride, void* q_out, const float* k_scale,
                            const float* v_scale, const void* q_weight, const void* k_weight, float eps,
                            const float* rope, int rope_rows, int rot_dim, int interleaved, const int32_t* cache_lens,
                            const int32_t* page_table, int max_blocks_per_seq, int num_blocks, int cache_capacity,
                            int B, int T, int Hq, int Hkv, int d, void* stream) {
  return append_norm_rope_impl(k_cache, v_cache, q, k_new, v_new, q_stride, k_stride, v_stride, q_out, k_scale, v_scale,
                               true, q_weight, k_weight, eps, rope, rope_rows, rot_dim, interleaved, cache_lens,
                               page_table, max_blocks_per_seq, num_blocks, cache_capacity, B, T, Hq, Hkv, d, stream,
                               "kv_append_norm_rope_fp8");
}

int rope_table_fill(float* table, int rows, int rot_dim, double theta, void* stream) {
  if (!table || rows < 1 || rot_dim < 2 || rot_dim % 2 || !(theta > 0.0) || !isfinite(theta))
    return ATTN_ERR_INVALID_ARG;
  return cuda_status(launch_rope_table(table, rows, rot_dim, theta, static_cast<cudaStream_t>(stream)),
                     "rope_table_fill");
}

}  // extern "C"
