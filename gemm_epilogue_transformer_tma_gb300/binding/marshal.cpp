// Argument marshalling of the entry points that serve single tokens or run
// many times per step, in C++: a launch takes 1.3 us on the host, the same
// tests of five tensors and a foreign call written in Python 3 to 5.
//
// Each function takes torch tensors (or None where the entry point takes
// NULL), extents and a stream (a torch stream, or None: the current one of the
// tensors' device), tests type, shape, contiguity and device, and calls the
// library entry point of the same name on the device's handle.  It returns the
// entry point's status.  The library's addresses come from bind(): this module
// does not link against it.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <initializer_list>

#include "../../include/coda.h"

namespace {

decltype(&coda_fp8_block_quantize) p_quantize;
decltype(&coda_fp8_block_quantize_weight) p_quantize_weight;
decltype(&coda_fp8_block_dequantize) p_dequantize;
decltype(&coda_gemm_fp8_block) p_gemm;
decltype(&coda_qknorm_rope) p_qknorm;
decltype(&coda_qknorm_rope_bwd) p_qknorm_bwd;
decltype(&coda_lmhead_policy) p_policy;
decltype(&coda_lmhead_score) p_score;
decltype(&coda_lmhead_distill) p_distill;

constexpr int kMaxDevices = 64;
coda_handle_t g_handles[kMaxDevices];
PyObject* g_make_handle;  // device index -> handle (an int)

constexpr auto BF = at::ScalarType::BFloat16;
constexpr auto F32 = at::ScalarType::Float;
constexpr auto I32 = at::ScalarType::Int;
constexpr auto U8 = at::ScalarType::Byte;

// One call's arguments; the first failure sets the Python error and every
// later step passes.
struct Call {
  PyObject* const* a;
  bool ok = true;
  int dev = -1;
  coda_handle_t handle = nullptr;
  void* stream = nullptr;

  Call(PyObject* const* args, Py_ssize_t given, Py_ssize_t wanted) : a(args) {
    if (given != wanted) {
      PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
      ok = false;
    }
  }
  const at::Tensor* tensor(int i, const char* name) {
    if (!ok) return nullptr;
    if (!THPVariable_Check(a[i])) {
      PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(a[i]);
  }
  // the device of argument i, its handle, and the stream argument s
  void on(int i, const char* name, int s) {
    const at::Tensor* t = tensor(i, name);
    if (t == nullptr) return;
    if (!t->is_cuda()) {
      PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
      ok = false;
      return;
    }
    dev = t->get_device();
    if (dev < 0 || dev >= kMaxDevices) {
      PyErr_SetString(PyExc_ValueError, "device index out of range");
      ok = false;
      return;
    }
    handle = g_handles[dev];
    if (handle == nullptr) {
      PyObject* h = PyObject_CallFunction(g_make_handle, "i", dev);
      handle = h == nullptr ? nullptr : static_cast<coda_handle_t>(PyLong_AsVoidPtr(h));
      Py_XDECREF(h);
      if (handle == nullptr) {
        ok = false;
        return;
      }
      g_handles[dev] = handle;
    }
    if (a[s] == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    } else {
      PyObject* p = PyObject_GetAttrString(a[s], "cuda_stream");
      if (p != nullptr) stream = PyLong_AsVoidPtr(p);
      Py_XDECREF(p);
      if (PyErr_Occurred()) ok = false;
    }
  }
  int64_t extent(int i, const char* name, int dim, int of) {
    const at::Tensor* t = tensor(i, name);
    if (t == nullptr) return 0;
    if (t->dim() != of) {
      PyErr_Format(PyExc_ValueError, "%s has %d dimensions, expected %d", name, static_cast<int>(t->dim()), of);
      ok = false;
      return 0;
    }
    return t->size(dim);
  }
  // the address of a contiguous tensor of that type and shape on the device
  void* arg(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(i, name);
    if (t == nullptr) return nullptr;
    PyObject* what = nullptr;
    const char* msg = nullptr;
    if (!t->is_cuda()) {
      what = PyExc_ValueError, msg = "%s must be a CUDA tensor";
    } else if (!t->is_contiguous()) {
      what = PyExc_ValueError, msg = "%s must be contiguous";
    } else if (t->scalar_type() != type) {
      what = PyExc_TypeError, msg = "%s has the wrong dtype";
    } else if (t->sizes() != c10::IntArrayRef(shape.begin(), shape.size())) {
      what = PyExc_ValueError, msg = "%s has the wrong shape";
    } else if (t->get_device() != dev) {
      what = PyExc_ValueError, msg = "%s is on another device than the other tensors";
    } else {
      return const_cast<void*>(t->const_data_ptr());
    }
    PyErr_Format(what, msg, name);
    ok = false;
    return nullptr;
  }
  void* opt(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return ok && a[i] != Py_None ? arg(i, name, type, shape) : nullptr;
  }
  // a workspace of any type and shape
  void* workspace(int i, size_t* bytes) {
    const at::Tensor* t = tensor(i, "ws");
    if (t == nullptr) return nullptr;
    *bytes = t->nbytes();
    if (!t->is_cuda() || !t->is_contiguous() || t->get_device() != dev) {
      PyErr_SetString(PyExc_ValueError, "ws must be a contiguous CUDA tensor on the other tensors' device");
      ok = false;
      return nullptr;
    }
    return const_cast<void*>(t->const_data_ptr());
  }
  int64_t num(int i) {
    if (!ok) return 0;
    const int64_t v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  int flag(int i) {
    if (!ok) return 0;
    const int v = PyObject_IsTrue(a[i]);
    if (v < 0) ok = false;
    return v;
  }
  float real(int i) {
    if (!ok) return 0.f;
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return static_cast<float>(v);
  }
};

// bytes of packed block scales (coda_fp8_block_scale_bytes)
int64_t packed(int64_t rows, int64_t K) { return (rows + 127) / 128 * ((K + 511) / 512) * 512; }

// f() without the interpreter lock, its status as a Python int
template <class F>
PyObject* finish(const Call& c, F&& f) {
  if (!c.ok) return nullptr;
  coda_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// (src, q_row, s_row, q_col, s_col, fmt, stream)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 7);
  c.on(0, "src", 6);
  const int64_t R = c.extent(0, "src", 0, 2), C = c.extent(0, "src", 1, 2);
  if (c.ok && ((a[1] == Py_None) != (a[2] == Py_None) || (a[3] == Py_None) != (a[4] == Py_None))) {
    PyErr_SetString(PyExc_ValueError, "codes and their scales come together");
    c.ok = false;
  }
  void* src = c.arg(0, "src", BF, {R, C});
  void* qr = c.opt(1, "q_row", U8, {R, C});
  void* sr = c.opt(2, "s_row", U8, {packed(R, C)});
  void* qc = c.opt(3, "q_col", U8, {R, C});
  void* sc = c.opt(4, "s_col", U8, {packed(C, R)});
  const int fmt = static_cast<int>(c.num(5));
  return finish(c, [&] { return p_quantize(c.handle, src, fmt, qr, sr, qc, sc, R, C, c.stream); });
}

// (W, q, s, s_t, fmt, stream)
PyObject* quantize_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 6);
  c.on(0, "W", 5);
  const int64_t N = c.extent(0, "W", 0, 2), K = c.extent(0, "W", 1, 2);
  void* W = c.arg(0, "W", BF, {N, K});
  void* q = c.arg(1, "q", U8, {N, K});
  void* s = c.arg(2, "s", U8, {packed(N, K)});
  void* st = c.arg(3, "s_t", U8, {packed(K, N)});
  const int fmt = static_cast<int>(c.num(4));
  return finish(c, [&] { return p_quantize_weight(c.handle, W, fmt, q, s, st, N, K, c.stream); });
}

// (q, s, col_blocks, dst, fmt, stream)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 6);
  c.on(0, "q", 5);
  const int64_t R = c.extent(0, "q", 0, 2), C = c.extent(0, "q", 1, 2);
  const int col = c.flag(2);
  void* q = c.arg(0, "q", U8, {R, C});
  void* s = c.arg(1, "s", U8, {col ? packed(C, R) : packed(R, C)});
  void* dst = c.arg(3, "dst", BF, {R, C});
  const int fmt = static_cast<int>(c.num(4));
  return finish(c, [&] { return p_dequantize(c.handle, q, s, col, fmt, dst, R, C, c.stream); });
}

// (A, a_mn_major, a_format, sA, B, b_mn_major, b_format, sB, C, M, N, K, stream)
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 13);
  c.on(8, "C", 12);
  const int64_t M = c.num(9), N = c.num(10), K = c.num(11);
  const int amn = c.flag(1), bmn = c.flag(5);
  const int fa = static_cast<int>(c.num(2)), fb = static_cast<int>(c.num(6));
  void* A = c.arg(0, "A", U8, {amn ? K : M, amn ? M : K});
  void* sA = c.arg(3, "sA", U8, {packed(M, K)});
  void* B = c.arg(4, "B", U8, {bmn ? K : N, bmn ? N : K});
  void* sB = c.arg(7, "sB", U8, {packed(N, K)});
  void* out = c.arg(8, "C", BF, {M, N});
  return finish(c, [&] { return p_gemm(c.handle, A, amn, fa, sA, B, bmn, fb, sB, out, M, N, K, c.stream); });
}

// (qkv, gq, gk, cos_t, sin_t, out, n_q_heads, n_kv_heads, head_dim, eps, positions, stream)
PyObject* qknorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 12);
  c.on(0, "qkv", 11);
  const int64_t M = c.extent(0, "qkv", 0, 2), S = c.extent(3, "cos_t", 0, 2);
  const int64_t nq = c.num(6), nkv = c.num(7), D = c.num(8);
  const int64_t W = (nq + 2 * nkv) * D;
  const float eps = c.real(9);
  void* x = c.arg(0, "qkv", BF, {M, W});
  void* gq = c.arg(1, "gq", BF, {D});
  void* gk = c.opt(2, "gk", BF, {D});
  auto* ct = static_cast<const float*>(c.arg(3, "cos_t", F32, {S, D / 2}));
  auto* sn = static_cast<const float*>(c.arg(4, "sin_t", F32, {S, D / 2}));
  void* out = c.arg(5, "out", BF, {M, W});
  auto* pos = static_cast<const int32_t*>(c.opt(10, "positions", I32, {M}));
  return finish(c, [&] { return p_qknorm(c.handle, x, gq, gk, ct, sn, pos, out, M, nq, nkv, D, S, eps, c.stream); });
}

// (dout, qkv, gq, gk, cos_t, sin_t, dqkv, dgq, dgk, ws, n_q_heads, n_kv_heads, head_dim, eps, positions, stream)
PyObject* qknorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 16);
  c.on(7, "dgq", 15);
  const int64_t M = c.extent(1, "qkv", 0, 2), S = c.extent(4, "cos_t", 0, 2);
  const int64_t nq = c.num(10), nkv = c.num(11), D = c.num(12);
  const int64_t W = (nq + 2 * nkv) * D;
  const float eps = c.real(13);
  size_t bytes = 0;
  void* dout = c.arg(0, "dout", BF, {M, W});
  void* x = c.arg(1, "qkv", BF, {M, W});
  void* gq = c.arg(2, "gq", BF, {D});
  void* gk = c.opt(3, "gk", BF, {D});
  auto* ct = static_cast<const float*>(c.arg(4, "cos_t", F32, {S, D / 2}));
  auto* sn = static_cast<const float*>(c.arg(5, "sin_t", F32, {S, D / 2}));
  void* dx = c.arg(6, "dqkv", BF, {M, W});
  auto* dgq = static_cast<float*>(c.arg(7, "dgq", F32, {D}));
  auto* dgk = static_cast<float*>(c.opt(8, "dgk", F32, {D}));
  void* ws = c.workspace(9, &bytes);
  auto* pos = static_cast<const int32_t*>(c.opt(14, "positions", I32, {M}));
  return finish(c, [&] {
    return p_qknorm_bwd(c.handle, dout, x, gq, gk, ct, sn, pos, dx, dgq, dgk, ws, bytes, M, nq, nkv, D, S, eps,
                        c.stream);
  });
}

// (Hs, Wt, labels, advantage, weight, logp_old, logp_ref, clip_low, clip_high, kl_coef, temperature, stats, logp,
//  dHs, dWt, ws, stream)
PyObject* policy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 17);
  c.on(0, "Hs", 16);
  const int64_t M = c.extent(0, "Hs", 0, 2), d = c.extent(0, "Hs", 1, 2), V = c.extent(1, "Wt", 0, 2);
  if (c.ok && (a[13] == Py_None) != (a[14] == Py_None)) {
    PyErr_SetString(PyExc_ValueError, "dHs and dWt come together");
    c.ok = false;
  }
  const float lo = c.real(7), hi = c.real(8), beta = c.real(9), T = c.real(10);
  size_t bytes = 0;
  void* H = c.arg(0, "Hs", BF, {M, d});
  void* W = c.arg(1, "Wt", BF, {V, d});
  auto* y = static_cast<const int32_t*>(c.arg(2, "labels", I32, {M}));
  auto* adv = static_cast<const float*>(c.arg(3, "advantage", F32, {M}));
  auto* w = static_cast<const float*>(c.opt(4, "weight", F32, {M}));
  auto* old = static_cast<const float*>(c.opt(5, "logp_old", F32, {M}));
  auto* ref = static_cast<const float*>(c.opt(6, "logp_ref", F32, {M}));
  auto* stats = static_cast<float*>(c.arg(11, "stats", F32, {4}));
  auto* logp = static_cast<float*>(c.arg(12, "logp", F32, {M}));
  void* dH = c.opt(13, "dHs", BF, {M, d});
  void* dW = c.opt(14, "dWt", BF, {V, d});
  void* ws = c.workspace(15, &bytes);
  return finish(c, [&] {
    return p_policy(c.handle, H, W, y, adv, w, old, ref, lo, hi, beta, T, stats, logp, dH, dW, ws, bytes, M, d, V,
                    c.stream);
  });
}

// (Hs, Wt, labels, temperature, logp, entropy, top_ids, top_logp, ws, stream)
PyObject* score(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 10);
  c.on(0, "Hs", 9);
  const int64_t M = c.extent(0, "Hs", 0, 2), d = c.extent(0, "Hs", 1, 2), V = c.extent(1, "Wt", 0, 2);
  if (c.ok && ((a[2] == Py_None) != (a[4] == Py_None) || (a[6] == Py_None) != (a[7] == Py_None))) {
    PyErr_SetString(PyExc_ValueError, "labels and logp, top_ids and top_logp come together");
    c.ok = false;
  }
  const int64_t k = c.ok && a[6] != Py_None ? c.extent(6, "top_ids", 1, 2) : 0;
  const float T = c.real(3);
  size_t bytes = 0;
  void* H = c.arg(0, "Hs", BF, {M, d});
  void* W = c.arg(1, "Wt", BF, {V, d});
  auto* y = static_cast<const int32_t*>(c.opt(2, "labels", I32, {M}));
  auto* logp = static_cast<float*>(c.opt(4, "logp", F32, {M}));
  auto* entropy = static_cast<float*>(c.opt(5, "entropy", F32, {M}));
  auto* ids = static_cast<int32_t*>(c.opt(6, "top_ids", I32, {M, k}));
  auto* top = static_cast<float*>(c.opt(7, "top_logp", F32, {M, k}));
  void* ws = c.workspace(8, &bytes);
  return finish(c, [&] {
    return p_score(c.handle, H, W, y, T, logp, entropy, ids, top, k, ws, bytes, M, d, V, c.stream);
  });
}

// (Hs, Wt, ids, val, weight, mode, temperature, stats, row_loss, dHs, dWt, ws, stream)
PyObject* distill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 13);
  c.on(0, "Hs", 12);
  const int64_t M = c.extent(0, "Hs", 0, 2), d = c.extent(0, "Hs", 1, 2), V = c.extent(1, "Wt", 0, 2);
  const int64_t k = c.extent(2, "ids", 1, 2);
  if (c.ok && (a[9] == Py_None) != (a[10] == Py_None)) {
    PyErr_SetString(PyExc_ValueError, "dHs and dWt come together");
    c.ok = false;
  }
  const int64_t mode = c.num(5);
  const float T = c.real(6);
  size_t bytes = 0;
  void* H = c.arg(0, "Hs", BF, {M, d});
  void* W = c.arg(1, "Wt", BF, {V, d});
  auto* ids = static_cast<const int32_t*>(c.arg(2, "ids", I32, {M, k}));
  auto* val = static_cast<const float*>(c.arg(3, "val", F32, {M, k}));
  auto* w = static_cast<const float*>(c.opt(4, "weight", F32, {M}));
  auto* stats = static_cast<float*>(c.arg(7, "stats", F32, {4}));
  auto* loss = static_cast<float*>(c.opt(8, "row_loss", F32, {M}));
  void* dH = c.opt(9, "dHs", BF, {M, d});
  void* dW = c.opt(10, "dWt", BF, {V, d});
  void* ws = c.workspace(11, &bytes);
  return finish(c, [&] {
    return p_distill(c.handle, H, W, ids, val, w, mode == static_cast<int>(mode) ? static_cast<int>(mode) : -1, T, stats,
                     loss, dH, dW, k, ws, bytes, M, d, V, c.stream);
  });
}

// bind(make_handle, quantize, quantize_weight, dequantize, gemm, qknorm, qknorm_bwd, policy, score, distill): the
// addresses of the library's entry points
constexpr int kBound = 10;
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, kBound);
  if (!c.ok) return nullptr;
  void* p[kBound] = {};
  for (int i = 1; i < kBound; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  Py_INCREF(a[0]);
  Py_XSETREF(g_make_handle, a[0]);
  p_quantize = reinterpret_cast<decltype(p_quantize)>(p[1]);
  p_quantize_weight = reinterpret_cast<decltype(p_quantize_weight)>(p[2]);
  p_dequantize = reinterpret_cast<decltype(p_dequantize)>(p[3]);
  p_gemm = reinterpret_cast<decltype(p_gemm)>(p[4]);
  p_qknorm = reinterpret_cast<decltype(p_qknorm)>(p[5]);
  p_qknorm_bwd = reinterpret_cast<decltype(p_qknorm_bwd)>(p[6]);
  p_policy = reinterpret_cast<decltype(p_policy)>(p[7]);
  p_score = reinterpret_cast<decltype(p_score)>(p[8]);
  p_distill = reinterpret_cast<decltype(p_distill)>(p[9]);
  Py_RETURN_NONE;
}

// A method as Python calls it: a C++ exception (a tensor without storage, a
// sparse one) becomes a Python one instead of crossing the C boundary.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

#define CODA_METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CODA_METHOD(bind),       CODA_METHOD(quantize), CODA_METHOD(quantize_weight),
                           CODA_METHOD(dequantize), CODA_METHOD(gemm),     CODA_METHOD(qknorm),
                           CODA_METHOD(qknorm_bwd), CODA_METHOD(policy),   CODA_METHOD(score),
                           CODA_METHOD(distill),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", "Argument marshalling of libcoda calls.", -1, g_methods,
                        nullptr,               nullptr, nullptr,                                nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
