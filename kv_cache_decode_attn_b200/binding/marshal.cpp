// Argument marshalling of the Python binding for the windowed, shared-prefix and
// norm-rotate-append calls: shape, type, device and contiguity checks of torch tensors,
// then the C call.  The calls' kernels take a few microseconds; through ctypes and Python
// the checks and conversions of about 25 arguments took 7 to 11 us of host time, here
// under 1 us.  Every function takes (device, stream handle, ...) positionally, returns the
// C call's status, and raises ValueError for arguments that do not fit.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "attn.h"

namespace {

using at::ScalarType;

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(const char* format, const char* what = "") {
  PyErr_Format(PyExc_ValueError, format, what);
  throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}

// Pointer of a tensor of device `dev`.
void* place(const at::Tensor& t, const char* name, int dev, bool contiguous = true) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  if (t.get_device() != dev) refuse("%s must be on the current device, like the other tensors", name);
  if (contiguous && !t.is_contiguous()) refuse("%s must be contiguous", name);
  return t.data_ptr();
}

void* typed(PyObject* o, const char* name, ScalarType type, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type) refuse("%s has the wrong dtype", name);
  return place(t, name, dev);
}

// None: no pointer.  An empty tensor has none either, so who asks for shapes asks for None, not for the pointer.
void* optional(PyObject* o, const char* name, ScalarType type, int dev) {
  return o == Py_None ? nullptr : typed(o, name, type, dev);
}

// A bf16 cache, or an FP8 one: e4m3 codes as uint8 or float8_e4m3fn.
void* cache(const at::Tensor& t, const char* name, bool fp8, int dev) {
  const ScalarType s = t.scalar_type();
  if (fp8 ? s != at::kByte && s != at::kFloat8_e4m3fn : s != at::kBFloat16) refuse("%s has the wrong dtype", name);
  return place(t, name, dev);
}

int out_type(const at::Tensor& o) {
  if (o.scalar_type() == at::kFloat) return ATTN_F32;
  if (o.scalar_type() == at::kBFloat16) return ATTN_BF16;
  refuse("output must be float32 or bfloat16");
}

int i32(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    if (PyErr_ExceptionMatches(PyExc_OverflowError)) refuse("value does not fit in 32 bits");
    throw Refused{};
  }
  if (v < INT32_MIN || v > INT32_MAX) refuse("value does not fit in 32 bits");
  return (int)v;
}

int dim(int64_t n) {
  if (n > INT32_MAX) refuse("a tensor's size does not fit in 32 bits");
  return (int)n;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return (float)v;
}

float scale_or_default(PyObject* o, int d) { return o == Py_None ? 1.f / std::sqrt((float)d) : real(o); }

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

void* stream_of(PyObject* o) { return PyLong_AsVoidPtr(o); }

// Other Python threads run while the C call launches (a launch may wait for queue space).
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

// q [B, T, Hq, d] and the output of its shape, lse [B, Hq, T] or none.
struct Queries {
  int B, T, Hq, d, o_type;
  void *q, *o;
  float* lse;
  Queries(PyObject* q_, PyObject* o_, PyObject* lse_, int dev) {
    const at::Tensor &tq = tensor(q_, "q"), &to = tensor(o_, "o");
    if (tq.dim() != 4 || to.sizes() != tq.sizes()) refuse("shape mismatch");
    B = dim(tq.size(0)), T = dim(tq.size(1)), Hq = dim(tq.size(2)), d = dim(tq.size(3));
    if (tq.scalar_type() != at::kBFloat16) refuse("%s has the wrong dtype", "q");
    q = place(tq, "q", dev);
    o = place(to, "o", dev);
    o_type = out_type(to);
    lse = static_cast<float*>(optional(lse_, "lse", at::kFloat, dev));
    if (lse_ != Py_None) {
      const at::Tensor& tl = THPVariable_Unpack(lse_);
      if (tl.dim() != 3 || tl.size(0) != B || tl.size(1) != Hq || tl.size(2) != T) refuse("lse must be [B, Hq, T]");
    }
  }
};

// The cache of B sequences: contiguous [B, capacity, Hkv, d], or pools [num_blocks, 16, Hkv, d] with a
// page table [B, max_blocks]; lengths [B]; FP8 (the call's say, not the arguments'): scales [Hkv].
struct Cache {
  int max_blocks = 0, num_blocks = 0, capacity = 0, Hkv;
  void *k, *v;
  float *k_scale = nullptr, *v_scale = nullptr;
  int32_t *lens, *table = nullptr;
  Cache(bool fp8, PyObject* k_, PyObject* v_, PyObject* ks_, PyObject* vs_, PyObject* lens_, PyObject* table_, int B,
        int d, int dev) {
    const at::Tensor &tk = tensor(k_, "k_cache"), &tv = tensor(v_, "v_cache"), &tl = tensor(lens_, "lengths");
    if (tk.dim() != 4 || tv.sizes() != tk.sizes() || tk.size(3) != d || tl.dim() != 1 || tl.size(0) != B)
      refuse("shape mismatch");
    Hkv = dim(tk.size(2));
    if (fp8) {
      const at::Tensor &ts = tensor(ks_, "k_scale"), &tw = tensor(vs_, "v_scale");
      if (ts.dim() != 1 || ts.size(0) != Hkv || tw.sizes() != ts.sizes()) refuse("k_scale and v_scale must be [Hkv]");
      k_scale = static_cast<float*>(typed(ks_, "k_scale", at::kFloat, dev));
      v_scale = static_cast<float*>(typed(vs_, "v_scale", at::kFloat, dev));
    }
    k = cache(tk, "k_cache", fp8, dev);
    v = cache(tv, "v_cache", fp8, dev);
    lens = static_cast<int32_t*>(typed(lens_, "lengths", at::kInt, dev));
    if (table_ == Py_None) {
      if (tk.size(0) != B) refuse("a contiguous cache must be [B, capacity, Hkv, d]");
      capacity = dim(tk.size(1));
      return;
    }
    const at::Tensor& tt = tensor(table_, "page_table");
    if (tk.size(1) != 16 || tt.dim() != 2 || tt.size(0) != B)
      refuse("a paged cache must be [num_blocks, 16, Hkv, d] with a page table [B, max_blocks]");
    table = static_cast<int32_t*>(typed(table_, "page_table", at::kInt, dev));
    max_blocks = dim(tt.size(1));
    num_blocks = dim(tk.size(0));
  }
};

struct Workspace {
  void* p;
  size_t n;
  Workspace(PyObject* o, int dev) {
    const at::Tensor& t = tensor(o, "workspace");
    p = place(t, "workspace", dev);
    n = t.nbytes();
  }
};

// Rows of B * T tokens, [B, T, H, d] bf16: each token's heads contiguous and the tokens evenly
// spaced -- contiguous, or a view of a fused projection output.
struct Rows {
  void* p;
  int64_t stride;
  Rows(PyObject* o, const char* name, int B, int T, int d, int dev) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 4 || t.size(0) != B || t.size(1) != T || t.size(3) != d) refuse("shape mismatch");
    if (t.scalar_type() != at::kBFloat16) refuse("%s has the wrong dtype", name);
    p = place(t, name, dev, false);
    const int64_t H = t.size(2);
    stride = T > 1 ? t.stride(1) : (B > 1 ? t.stride(0) : H * d);
    if ((d > 1 && t.stride(3) != 1) || (H > 1 && t.stride(2) != d) || (B > 1 && T > 1 && t.stride(0) != T * t.stride(1)))
      refuse("%s: each token's heads must be contiguous and the tokens evenly spaced", name);
  }
};

// q_weight, k_weight [d] and the angle table [rows, rot_dim], each or none.
struct Turn {
  void *qw, *kw;
  float* rope;
  int rows = 0, rot = 0;
  Turn(PyObject* qw_, PyObject* kw_, PyObject* rope_, int d, int dev) {
    qw = optional(qw_, "q_weight", at::kBFloat16, dev);
    kw = optional(kw_, "k_weight", at::kBFloat16, dev);
    for (PyObject* w : {qw_, kw_})
      if (w != Py_None && (THPVariable_Unpack(w).dim() != 1 || THPVariable_Unpack(w).size(0) != d))
        refuse("q_weight and k_weight must be [d]");
    rope = static_cast<float*>(optional(rope_, "rope", at::kFloat, dev));
    if (rope_ != Py_None) {
      const at::Tensor& t = THPVariable_Unpack(rope_);
      if (t.dim() != 2 || t.numel() == 0) refuse("rope must be [rows, rot_dim]");
      rows = dim(t.size(0));
      rot = dim(t.size(1));
    }
  }
};

// (dev, stream, q, k, v, o, window, sinks, lse, scale)
int prefill_window(PyObject* const* a) {
  const int dev = i32(a[0]);
  const Queries q(a[2], a[5], a[8], dev);
  const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
  if (k.dim() != 4 || k.size(0) != q.B || k.size(1) != q.T || k.size(3) != q.d || v.sizes() != k.sizes())
    refuse("shape mismatch");
  const void *kp = typed(a[3], "k", at::kBFloat16, dev), *vp = typed(a[4], "v", at::kBFloat16, dev);
  const int Hkv = dim(k.size(2)), window = i32(a[6]), sinks = i32(a[7]);
  const float scale = scale_or_default(a[9], q.d);
  void* stream = stream_of(a[1]);
  const NoGil free;
  return attn_prefill_window(q.q, kp, vp, q.o, q.o_type, q.lse, q.B, q.Hq, Hkv, q.T, q.d, scale, window, sinks, stream);
}

// (dev, stream, q, k_cache, v_cache, seqlens, o, window, sinks, lse, page_table, scale)
int prefill_cache_window(PyObject* const* a) {
  const int dev = i32(a[0]);
  const Queries q(a[2], a[6], a[9], dev);
  const Cache c(false, a[3], a[4], Py_None, Py_None, a[5], a[10], q.B, q.d, dev);
  const int window = i32(a[7]), sinks = i32(a[8]);
  const float scale = scale_or_default(a[11], q.d);
  void* stream = stream_of(a[1]);
  const NoGil free;
  return attn_prefill_cache_window(q.q, c.k, c.v, c.lens, c.table, c.max_blocks, c.num_blocks, c.capacity, q.o,
                                   q.o_type, q.lse, q.B, q.T, q.Hq, c.Hkv, q.d, scale, window, sinks, stream);
}

// (dev, stream, q, k_cache, v_cache, k_scale, v_scale, seqlens, o, window, sinks, lse, page_table, max_seqlen_k,
//  scale, num_splits, workspace)
template <bool FP8>
int decode_window(PyObject* const* a) {
  const int dev = i32(a[0]);
  const Queries q(a[2], a[8], a[11], dev);
  const Cache c(FP8, a[3], a[4], a[5], a[6], a[7], a[12], q.B, q.d, dev);
  const Workspace w(a[16], dev);
  const int window = i32(a[9]), sinks = i32(a[10]), longest = i32(a[13]), splits = i32(a[15]);
  const float scale = scale_or_default(a[14], q.d);
  void* stream = stream_of(a[1]);
  const NoGil free;
  if (FP8)
    return attn_decode_window_fp8(q.q, c.k, c.v, c.k_scale, c.v_scale, c.lens, c.table, c.max_blocks, c.num_blocks,
                                  c.capacity, longest, q.o, q.o_type, q.lse, q.B, q.T, q.Hq, c.Hkv, q.d, scale, window,
                                  sinks, splits, w.p, w.n, stream);
  return attn_decode_window(q.q, c.k, c.v, c.lens, c.table, c.max_blocks, c.num_blocks, c.capacity, longest, q.o,
                            q.o_type, q.lse, q.B, q.T, q.Hq, c.Hkv, q.d, scale, window, sinks, splits, w.p, w.n,
                            stream);
}

// (dev, stream, q, k_cache, v_cache, k_scale, v_scale, seqlens, page_table, prefix_table, o, lse, max_seqlen_k,
//  scale, causal, num_splits, workspace)
template <bool FP8>
int decode_shared(PyObject* const* a) {
  const int dev = i32(a[0]);
  if (a[8] == Py_None) refuse("a shared prefix needs a page table");
  const Queries q(a[2], a[10], a[11], dev);
  const Cache c(FP8, a[3], a[4], a[5], a[6], a[7], a[8], q.B, q.d, dev);
  const at::Tensor& prefix = tensor(a[9], "prefix_table");
  if (prefix.dim() != 1) refuse("prefix_table must be [prefix_blocks]");
  const int n = dim(prefix.size(0));
  const int32_t* pre = n ? static_cast<int32_t*>(typed(a[9], "prefix_table", at::kInt, dev)) : nullptr;
  const Workspace w(a[16], dev);
  const int longest = i32(a[12]), causal = truth(a[14]), splits = i32(a[15]);
  const float scale = scale_or_default(a[13], q.d);
  void* stream = stream_of(a[1]);
  const NoGil free;
  if (FP8)
    return attn_decode_shared_fp8(q.q, c.k, c.v, c.k_scale, c.v_scale, c.lens, c.table, c.max_blocks, c.num_blocks,
                                  pre, n, longest, q.o, q.o_type, q.lse, q.B, q.T, q.Hq, c.Hkv, q.d, scale, causal,
                                  splits, w.p, w.n, stream);
  return attn_decode_shared(q.q, c.k, c.v, c.lens, c.table, c.max_blocks, c.num_blocks, pre, n, longest, q.o, q.o_type,
                            q.lse, q.B, q.T, q.Hq, c.Hkv, q.d, scale, causal, splits, w.p, w.n, stream);
}

// (dev, stream, q, k, q_out, k_out, rope, q_weight, k_weight, eps, interleaved, pos0)
int norm_rope(PyObject* const* a) {
  const int dev = i32(a[0]);
  const at::Tensor &tq = tensor(a[2], "q"), &tk = tensor(a[3], "k");
  if (tq.dim() != 4 || tk.dim() != 4 || tensor(a[4], "q_out").sizes() != tq.sizes() ||
      tensor(a[5], "k_out").sizes() != tk.sizes())
    refuse("shape mismatch");
  const int B = dim(tq.size(0)), T = dim(tq.size(1)), Hq = dim(tq.size(2)), d = dim(tq.size(3));
  const Rows q(a[2], "q", B, T, d, dev), k(a[3], "k", B, T, d, dev);
  const Turn t(a[7], a[8], a[6], d, dev);
  const int32_t* pos0 = static_cast<int32_t*>(optional(a[11], "pos0", at::kInt, dev));
  if (a[11] != Py_None && (THPVariable_Unpack(a[11]).dim() != 1 || THPVariable_Unpack(a[11]).size(0) != B))
    refuse("pos0 must be [B]");
  void *q_out = typed(a[4], "q_out", at::kBFloat16, dev), *k_out = typed(a[5], "k_out", at::kBFloat16, dev);
  const int Hkv = dim(tk.size(2)), interleaved = truth(a[10]);
  const float eps = real(a[9]);
  void* stream = stream_of(a[1]);
  const NoGil free;
  return qk_norm_rope(q.p, k.p, q.stride, k.stride, q_out, k_out, t.qw, t.kw, eps, t.rope, t.rows, t.rot, interleaved,
                      pos0, B, T, Hq, Hkv, d, stream);
}

// (dev, stream, k_cache, v_cache, q, k_new, v_new, q_out, k_scale, v_scale, rope, cache_lens, page_table, q_weight,
//  k_weight, eps, interleaved)
template <bool FP8>
int append_norm_rope(PyObject* const* a) {
  const int dev = i32(a[0]);
  const at::Tensor &tq = tensor(a[4], "q"), &tk = tensor(a[5], "k_new"), &tv = tensor(a[6], "v_new");
  if (tq.dim() != 4 || tk.dim() != 4 || tv.sizes() != tk.sizes() || tensor(a[7], "q_out").sizes() != tq.sizes())
    refuse("shape mismatch");
  const int B = dim(tq.size(0)), T = dim(tq.size(1)), Hq = dim(tq.size(2)), d = dim(tq.size(3));
  const Cache c(FP8, a[2], a[3], a[8], a[9], a[11], a[12], B, d, dev);
  if (tk.size(2) != c.Hkv) refuse("shape mismatch");
  const Rows q(a[4], "q", B, T, d, dev), k(a[5], "k_new", B, T, d, dev), v(a[6], "v_new", B, T, d, dev);
  const Turn t(a[13], a[14], a[10], d, dev);
  void* q_out = typed(a[7], "q_out", at::kBFloat16, dev);
  const float eps = real(a[15]);
  const int interleaved = truth(a[16]);
  void* stream = stream_of(a[1]);
  const NoGil free;
  if (FP8)
    return kv_append_norm_rope_fp8(c.k, c.v, q.p, k.p, v.p, q.stride, k.stride, v.stride, q_out, c.k_scale, c.v_scale,
                                   t.qw, t.kw, eps, t.rope, t.rows, t.rot, interleaved, c.lens, c.table, c.max_blocks,
                                   c.num_blocks, c.capacity, B, T, Hq, c.Hkv, d, stream);
  return kv_append_norm_rope(c.k, c.v, q.p, k.p, v.p, q.stride, k.stride, v.stride, q_out, t.qw, t.kw, eps, t.rope,
                             t.rows, t.rot, interleaved, c.lens, c.table, c.max_blocks, c.num_blocks, c.capacity, B, T,
                             Hq, c.Hkv, d, stream);
}

template <int (*F)(PyObject* const*), int kArgs>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", kArgs, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

#define FAST(name, function, args) {name, (PyCFunction)(void (*)(void))call<function, args>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("prefill_window", prefill_window, 10),
                         FAST("prefill_cache_window", prefill_cache_window, 12),
                         FAST("decode_window", decode_window<false>, 17),
                         FAST("decode_window_fp8", decode_window<true>, 17),
                         FAST("decode_shared", decode_shared<false>, 17),
                         FAST("decode_shared_fp8", decode_shared<true>, 17),
                         FAST("norm_rope", norm_rope, 12),
                         FAST("append_norm_rope", append_norm_rope<false>, 17),
                         FAST("append_norm_rope_fp8", append_norm_rope<true>, 17),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&module);
  // the torch and Python whose headers this was compiled against
  if (m && PyModule_AddStringConstant(m, "built_for", KVATTN_BUILT_FOR)) Py_CLEAR(m);
  return m;
}
