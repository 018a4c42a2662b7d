// Short host path of the Python binding's few-token, FP8 and gradient calls (a CPython extension
// module; no device code).
//
// These calls can run a few microseconds on the GPU, and checking a dozen tensors and
// allocating the results from Python takes longer than that.  Each function here does
// for plain torch.Tensor arguments what its namesake in moe_fp4.py does: the same
// checks, the same allocations, the same call of the C entry point.  Where anything is
// out of the ordinary (another type, a failed check, an error status, an exception) it
// returns None without having enqueued anything, and the Python code runs, which names
// what is wrong.  The entry points' addresses come from the loaded library (bind).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_fp4.h"

namespace {

decltype(&moe_fp4_linear) g_linear;
decltype(&moe_fp4_ffn) g_ffn;
decltype(&moe_fp4_ffn_workspace_size) g_ffn_workspace;
decltype(&moe_fp4_route) g_route;
decltype(&moe_fp4_route_workspace_size) g_route_workspace;
decltype(&moe_fp8_quantize) g_quantize_fp8;
decltype(&moe_grouped_gemm_fp8) g_gemm_fp8;
decltype(&moe_fp4_dispatch) g_dispatch;
decltype(&moe_fp4_dispatch_backward) g_dispatch_backward;
decltype(&moe_fp4_combine_backward) g_combine_backward;
decltype(&moe_fp4_route_backward) g_route_backward;

// What makes a call leave for the Python code.
struct Leave {};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_CheckTypeExact(Py_TYPE(o))) throw Leave{};
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided) throw Leave{};
  return t;
}

// The device every tensor of a call is on.
struct Device {
  int index = -1;
  void add(const at::Tensor& t) {
    const int d = t.get_device();
    if (index >= 0 && d != index) throw Leave{};
    index = d;
  }
};

void need(bool ok) {
  if (!ok) throw Leave{};
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Leave{};
  return v;
}

// A contiguous tensor of this type and shape; returns its address.
void* exact(PyObject* o, at::ScalarType type, at::IntArrayRef shape, Device& dev) {
  const at::Tensor& t = tensor(o);
  need(t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
  dev.add(t);
  return t.data_ptr();
}

// A matrix with unit column stride: its pitch.
int64_t pitch(const at::Tensor& t, int64_t rows, int64_t cols) {
  need(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && (t.stride(1) == 1 || cols <= 1));
  return rows > 1 ? t.stride(0) : cols;
}

int in_code(at::ScalarType t) {
  if (t == at::kBFloat16) return MOE_FP4_IN_BF16;
  if (t == at::kFloat) return MOE_FP4_IN_FP32;
  need(t == at::kHalf);
  return MOE_FP4_IN_FP16;
}

int out_code(at::ScalarType t) {
  if (t == at::kBFloat16) return MOE_FP4_OUT_BF16;
  if (t == at::kFloat) return MOE_FP4_OUT_FP32;
  need(t == at::kHalf);
  return MOE_FP4_OUT_FP16;
}

// Activations, residual and output of a few-token call.
struct Rows {
  const void* x;
  const void* residual = nullptr;
  int64_t ld_x, ld_res = 0, ldo;
  int x_dtype, out_dtype;
  at::Tensor out;

  // The given output, or the new one.
  PyObject* result(PyObject* out_arg) const {
    if (out_arg == Py_None) return THPVariable_Wrap(out);
    Py_INCREF(out_arg);
    return out_arg;
  }

  // o_type: the output's type as MOE_FP4_OUT_*, -1 for x's.
  Rows(const at::Tensor& xt, PyObject* res, PyObject* out_arg, int64_t o_type, int64_t m, int64_t k,
       int64_t cols, Device& dev) {
    need(xt.scalar_type() == at::kBFloat16 || xt.scalar_type() == at::kHalf);
    dev.add(xt);
    x = xt.data_ptr();
    x_dtype = in_code(xt.scalar_type());
    ld_x = pitch(xt, m, k);
    if (res != Py_None) {
      const at::Tensor& r = tensor(res);
      need(r.scalar_type() == xt.scalar_type());
      dev.add(r);
      ld_res = pitch(r, m, cols);
      residual = r.data_ptr();
    }
    if (out_arg != Py_None) {
      out = tensor(out_arg);
      dev.add(out);
      out_dtype = out_code(out.scalar_type());
      need(o_type < 0 || o_type == out_dtype);
      ldo = pitch(out, m, cols);
    } else {
      const at::ScalarType types[] = {at::kBFloat16, at::kFloat, at::kHalf};
      need(o_type < 3);
      out = at::empty({m, cols}, xt.options().dtype(o_type < 0 ? xt.scalar_type() : types[o_type]));
      out_dtype = out_code(out.scalar_type());
      ldo = cols;
    }
  }
};

// (device index -> stream handle) as the caller found them; the tensors must be there.
void* stream_on(PyObject* device, PyObject* handle, const Device& dev) {
  need(integer(device) == dev.index);
  return reinterpret_cast<void*>(static_cast<intptr_t>(integer(handle)));
}

// Call an entry point without the interpreter lock (as ctypes does): a launch may wait
// for room in its queue.
template <typename F>
int unlocked(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(s);
  return status;
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kEntries = 11;
  if (n != kEntries) {
    PyErr_SetString(PyExc_TypeError, "bind: eleven addresses");
    return nullptr;
  }
  uintptr_t p[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    p[i] = (uintptr_t)PyLong_AsUnsignedLongLong(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
  g_ffn = reinterpret_cast<decltype(g_ffn)>(p[1]);
  g_ffn_workspace = reinterpret_cast<decltype(g_ffn_workspace)>(p[2]);
  g_route = reinterpret_cast<decltype(g_route)>(p[3]);
  g_route_workspace = reinterpret_cast<decltype(g_route_workspace)>(p[4]);
  g_quantize_fp8 = reinterpret_cast<decltype(g_quantize_fp8)>(p[5]);
  g_gemm_fp8 = reinterpret_cast<decltype(g_gemm_fp8)>(p[6]);
  g_dispatch = reinterpret_cast<decltype(g_dispatch)>(p[7]);
  g_dispatch_backward = reinterpret_cast<decltype(g_dispatch_backward)>(p[8]);
  g_combine_backward = reinterpret_cast<decltype(g_combine_backward)>(p[9]);
  g_route_backward = reinterpret_cast<decltype(g_route_backward)>(p[10]);
  Py_RETURN_NONE;
}

// linear(x, w_q, w_sf, w_scale, swiglu, residual, out, out_type, device, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 10 && g_linear);
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]);
    need(x.dim() == 2 && w.dim() == 2 && w.scalar_type() == at::kByte && w.is_contiguous());
    const int64_t m = x.size(0), k = x.size(1), rows = w.size(0);
    need(w.size(1) == k / 2 && k % 2 == 0);
    Device dev;
    dev.add(w);
    const int swiglu = PyObject_IsTrue(a[4]);
    need(swiglu >= 0 && !(swiglu && (rows % 2 != 0 || a[5] != Py_None)));
    const void* sf = exact(a[2], at::kByte, {rows, k / 16}, dev);
    const void* scale = exact(a[3], at::kFloat, {1}, dev);
    const Rows r(x, a[5], a[6], integer(a[7]), m, k, swiglu ? rows / 2 : rows, dev);
    void* stream = stream_on(a[8], a[9], dev);
    const int status = unlocked([&] {
      return g_linear(r.x, r.x_dtype, m, r.ld_x, static_cast<const uint8_t*>(w.data_ptr()),
                      static_cast<const uint8_t*>(sf), static_cast<const float*>(scale), rows, k, swiglu,
                      r.residual, r.ld_res, r.out.data_ptr(), r.out_dtype, r.ldo, stream);
    });
    need(status == MOE_FP4_OK);
    return r.result(a[6]);
  });
}

// ffn(x, ids, weights, w13_q, w13_sf, w13_scale, w2_q, w2_sf, w2_scale, residual, out,
//     out_type, device, stream): with a workspace of its own, on the current stream
PyObject* ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 14 && g_ffn);
    const at::Tensor &x = tensor(a[0]), &ids = tensor(a[1]), &w13 = tensor(a[3]);
    need(x.dim() == 2 && ids.dim() == 2 && w13.dim() == 3);
    const int64_t T = x.size(0), H = x.size(1), K = ids.size(1), E = w13.size(0), I = w13.size(1) / 2;
    need(H % 2 == 0 && I % 2 == 0 && E <= INT32_MAX && K <= INT32_MAX);
    Device dev;
    const void* idp = exact(a[1], at::kInt, {T, K}, dev);
    const void* wts = exact(a[2], at::kFloat, {T, K}, dev);
    const void* w13q = exact(a[3], at::kByte, {E, 2 * I, H / 2}, dev);
    const void* w13s = exact(a[4], at::kByte, {E, 2 * I, H / 16}, dev);
    const void* w13t = exact(a[5], at::kFloat, {E}, dev);
    const void* w2q = exact(a[6], at::kByte, {E, H, I / 2}, dev);
    const void* w2s = exact(a[7], at::kByte, {E, H, I / 16}, dev);
    const void* w2t = exact(a[8], at::kFloat, {E}, dev);
    const Rows r(x, a[9], a[10], integer(a[11]), T, H, H, dev);
    void* stream = stream_on(a[12], a[13], dev);
    const size_t bytes = g_ffn_workspace(T, (int32_t)K, (int32_t)E, I);
    const at::Tensor ws = at::empty({(int64_t)bytes}, w13.options());
    const int status = unlocked([&] {
      return g_ffn(r.x, r.x_dtype, T, r.ld_x, static_cast<const int32_t*>(idp), static_cast<const float*>(wts),
                   (int32_t)K, static_cast<const uint8_t*>(w13q), static_cast<const uint8_t*>(w13s),
                   static_cast<const float*>(w13t), static_cast<const uint8_t*>(w2q),
                   static_cast<const uint8_t*>(w2s), static_cast<const float*>(w2t), (int32_t)E, H, I,
                   r.residual, r.ld_res, r.out.data_ptr(), r.out_dtype, r.ldo, ws.data_ptr(), bytes, stream);
    });
    need(status == MOE_FP4_OK);
    return r.result(a[10]);
  });
}

// Elements (of four bytes) a result takes of a common allocation: whole 256 bytes.
int64_t aligned_part(int64_t n) { return (n + 63) / 64 * 64; }

// A contiguous tensor of four-byte elements at element `at` of another's storage.
at::Tensor part_of(const at::Tensor& all, at::ScalarType type, int64_t at, at::IntArrayRef shape) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                          c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// route(logits, topk, score, bias, renormalize, num_groups, topk_groups, device, stream):
// new outputs, a workspace of its own, on the current stream; a tuple of five tensors
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 9 && g_route);
    const at::Tensor& x = tensor(a[0]);
    need(x.dim() == 2);
    const int64_t T = x.size(0), E = x.size(1), K = integer(a[1]);
    need(K >= 1 && K <= INT32_MAX && E <= INT32_MAX);
    Device dev;
    dev.add(x);
    const int64_t ld = pitch(x, T, E);
    const int dtype = in_code(x.scalar_type());
    const void* logits = x.data_ptr();
    const void* bias = a[3] == Py_None ? nullptr : exact(a[3], at::kFloat, {E}, dev);
    const int renormalize = PyObject_IsTrue(a[4]);
    const int64_t score = integer(a[2]), groups = integer(a[5]), topk_groups = integer(a[6]);
    need(renormalize >= 0 && groups <= INT32_MAX && topk_groups <= INT32_MAX && groups >= 1 && topk_groups >= 1);
    void* stream = stream_on(a[7], a[8], dev);
    need(T <= INT32_MAX && T * K <= INT32_MAX);
    // One allocation for the five results: each allocation costs a tenth of a short call.
    const int64_t part = aligned_part(T * K), last = aligned_part(E + 1);
    const at::Tensor all = at::empty({4 * part + last}, x.options().dtype(at::kInt));
    const at::Tensor ids = part_of(all, at::kInt, 0, {T, K}), weights = part_of(all, at::kFloat, part, {T, K}),
                     row_token = part_of(all, at::kInt, 2 * part, {T * K}),
                     token_rows = part_of(all, at::kInt, 3 * part, {T, K}),
                     offsets = part_of(all, at::kInt, 4 * part, {E + 1});
    const size_t bytes = g_route_workspace(T, (int32_t)E);
    at::Tensor ws;
    if (bytes) ws = at::empty({(int64_t)bytes}, x.options().dtype(at::kByte));
    const int status = unlocked([&] {
      return g_route(logits, dtype, T, (int32_t)E, ld, (int)score,
                     static_cast<const float*>(bias), renormalize, (int32_t)K, (int32_t)groups,
                     (int32_t)topk_groups, static_cast<int32_t*>(ids.data_ptr()),
                     static_cast<float*>(weights.data_ptr()), static_cast<int32_t*>(offsets.data_ptr()),
                     static_cast<int32_t*>(row_token.data_ptr()), static_cast<int32_t*>(token_rows.data_ptr()),
                     bytes ? ws.data_ptr() : nullptr, bytes, stream);
    });
    need(status == MOE_FP4_OK);
    PyObject* out = PyTuple_New(5);
    if (!out) return nullptr;
    const at::Tensor* parts[] = {&ids, &weights, &offsets, &row_token, &token_rows};
    for (int i = 0; i < 5; ++i) {
      PyObject* t = THPVariable_Wrap(*parts[i]);
      if (!t) return Py_DECREF(out), nullptr;
      PyTuple_SET_ITEM(out, i, t);
    }
    return out;
  });
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// A matrix of one of the router's input types, with its pitch.
struct Matrix {
  const at::Tensor& t;
  int64_t rows, cols, ld;
  int dtype;
  Matrix(PyObject* o, Device& dev, bool fp8 = false) : t(tensor(o)) {
    need(t.dim() == 2);
    rows = t.size(0);
    cols = t.size(1);
    dtype = fp8 && t.scalar_type() == at::kFloat8_e4m3fn ? MOE_FP4_IN_FP8 : in_code(t.scalar_type());
    dev.add(t);
    ld = pitch(t, rows, cols);
  }
};

const int32_t* ints(void* p) { return static_cast<const int32_t*>(p); }

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* out = PyTuple_New(2);
  if (!out) return nullptr;
  const at::Tensor* parts[] = {&a, &b};
  for (int i = 0; i < 2; ++i) {
    PyObject* t = THPVariable_Wrap(*parts[i]);
    if (!t) return Py_DECREF(out), nullptr;
    PyTuple_SET_ITEM(out, i, t);
  }
  return out;
}

// quantize_fp8(x, swiglu, grad, power_of_two, device, stream): new outputs
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 6 && g_quantize_fp8);
    Device dev;
    const Matrix x(a[0], dev);
    const int swiglu = PyObject_IsTrue(a[1]), pow2 = PyObject_IsTrue(a[3]);
    need(swiglu >= 0 && pow2 >= 0 && !(swiglu && x.cols % 2 != 0));
    const int64_t k = swiglu ? x.cols / 2 : x.cols;
    const void* grad = nullptr;
    int64_t ld_grad = 0;
    if (a[2] != Py_None) {
      const Matrix g(a[2], dev);
      need(swiglu && g.dtype == x.dtype && g.rows == x.rows && g.cols == k);
      grad = g.t.data_ptr();
      ld_grad = g.ld;
    }
    void* stream = stream_on(a[4], a[5], dev);
    const int64_t cols = grad ? x.cols : k;
    const at::Tensor q = at::empty({x.rows, cols}, x.t.options().dtype(at::kFloat8_e4m3fn));
    const at::Tensor sf = at::empty({x.rows, blocks(cols)}, x.t.options().dtype(at::kFloat));
    const int status = unlocked([&] {
      return g_quantize_fp8(x.t.data_ptr(), x.dtype, x.rows, k, x.ld, swiglu, grad, ld_grad, pow2,
                            static_cast<uint8_t*>(q.data_ptr()), static_cast<float*>(sf.data_ptr()), stream);
    });
    need(status == MOE_FP4_OK);
    return pair(q, sf);
  });
}

// gemm_fp8(a_q, a_sf, w_q, w_sf, offsets, a_row_index, out_type, device, stream): a new output;
// offsets None: one expert, w_q [n][k]
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 9 && g_gemm_fp8);
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[2]);
    const bool dense = a[4] == Py_None;
    need(x.dim() == 2 && w.dim() == (dense ? 2 : 3));
    const int64_t rows = x.size(0), k = x.size(1), E = dense ? 1 : w.size(0), N = w.size(dense ? 0 : 1);
    need(E <= INT32_MAX);
    Device dev;
    const void* xq = exact(a[0], at::kFloat8_e4m3fn, {rows, k}, dev);
    const void* xs = exact(a[1], at::kFloat, {rows, blocks(k)}, dev);
    const void *wq, *ws, *off = nullptr, *index = nullptr;
    if (dense) {
      wq = exact(a[2], at::kFloat8_e4m3fn, {N, k}, dev);
      ws = exact(a[3], at::kFloat, {blocks(N), blocks(k)}, dev);
    } else {
      wq = exact(a[2], at::kFloat8_e4m3fn, {E, N, k}, dev);
      ws = exact(a[3], at::kFloat, {E, blocks(N), blocks(k)}, dev);
      off = exact(a[4], at::kInt, {E + 1}, dev);
    }
    int64_t m = rows;
    if (a[5] != Py_None) {
      m = tensor(a[5]).numel();
      index = exact(a[5], at::kInt, {m}, dev);
    }
    const int64_t type = integer(a[6]);
    need(type >= 0 && type < 3);
    void* stream = stream_on(a[7], a[8], dev);
    const at::ScalarType types[] = {at::kBFloat16, at::kFloat, at::kHalf};
    const at::Tensor out = at::empty({m, N}, x.options().dtype(types[type]));
    const int status = unlocked([&] {
      return g_gemm_fp8(static_cast<const uint8_t*>(xq), static_cast<const float*>(xs), rows,
                        static_cast<const int32_t*>(index), static_cast<const uint8_t*>(wq),
                        static_cast<const float*>(ws), static_cast<const int32_t*>(off), (int32_t)E, m, N, k,
                        out.data_ptr(), (int)type, N, stream);
    });
    need(status == MOE_FP4_OK);
    return THPVariable_Wrap(out);
  });
}

// dispatch(x, row_token, device, stream): a new output
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 4 && g_dispatch);
    Device dev;
    const Matrix x(a[0], dev, true);
    const int64_t m = tensor(a[1]).numel();
    void* map = exact(a[1], at::kInt, {m}, dev);
    void* stream = stream_on(a[2], a[3], dev);
    const at::Tensor out = at::empty({m, x.cols}, x.t.options());
    const int status = unlocked([&] {
      return g_dispatch(x.t.data_ptr(), x.dtype, x.rows, x.cols, x.ld, ints(map), m, out.data_ptr(), x.cols, stream);
    });
    need(status == MOE_FP4_OK);
    return THPVariable_Wrap(out);
  });
}

// dispatch_backward(dy, token_rows, device, stream): a new output
PyObject* dispatch_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 4 && g_dispatch_backward);
    Device dev;
    const Matrix y(a[0], dev);
    const at::Tensor& rows = tensor(a[1]);
    need(rows.dim() == 2);
    const int64_t T = rows.size(0), K = rows.size(1);
    need(K >= 1 && K <= INT32_MAX);
    void* map = exact(a[1], at::kInt, {T, K}, dev);
    void* stream = stream_on(a[2], a[3], dev);
    const at::Tensor out = at::empty({T, y.cols}, y.t.options());
    const int status = unlocked([&] {
      return g_dispatch_backward(y.t.data_ptr(), y.dtype, y.rows, y.cols, y.ld, ints(map), (int32_t)K, T,
                                 out.data_ptr(), y.cols, stream);
    });
    need(status == MOE_FP4_OK);
    return THPVariable_Wrap(out);
  });
}

// combine_backward(dout, rows, token_rows, token_weights, row_token, device, stream): new outputs
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 7 && g_combine_backward);
    Device dev;
    const Matrix g(a[0], dev), r(a[1], dev);
    need(g.dtype != MOE_FP4_IN_FP16 && r.dtype == MOE_FP4_IN_BF16 && r.cols == g.cols);
    const at::Tensor& map = tensor(a[2]);
    need(map.dim() == 2 && map.size(0) == g.rows);
    const int64_t K = map.size(1);
    need(K >= 1 && K <= INT32_MAX);
    void* rows = exact(a[2], at::kInt, {g.rows, K}, dev);
    const void* weights = exact(a[3], at::kFloat, {g.rows, K}, dev);
    void* row_token = exact(a[4], at::kInt, {r.rows}, dev);
    void* stream = stream_on(a[5], a[6], dev);
    const at::Tensor drows = at::empty({r.rows, r.cols}, r.t.options());
    const at::Tensor dweights = at::empty({g.rows, K}, g.t.options().dtype(at::kFloat));
    const int status = unlocked([&] {
      return g_combine_backward(g.t.data_ptr(), g.dtype == MOE_FP4_IN_FP32 ? MOE_FP4_OUT_FP32 : MOE_FP4_OUT_BF16,
                                g.rows, g.cols, g.ld, static_cast<const uint16_t*>(r.t.data_ptr()), r.ld, r.rows,
                                ints(rows), static_cast<const float*>(weights), (int32_t)K, ints(row_token),
                                static_cast<uint16_t*>(drows.data_ptr()), r.cols,
                                static_cast<float*>(dweights.data_ptr()), stream);
    });
    need(status == MOE_FP4_OK);
    return pair(drows, dweights);
  });
}

// route_backward(logits, ids, dweights, score, renormalize, device, stream): a new output
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 7 && g_route_backward);
    Device dev;
    const Matrix x(a[0], dev);
    const at::Tensor& idt = tensor(a[1]);
    need(idt.dim() == 2 && idt.size(0) == x.rows && x.cols <= INT32_MAX);
    const int64_t K = idt.size(1);
    need(K >= 1 && K <= INT32_MAX);
    void* ids = exact(a[1], at::kInt, {x.rows, K}, dev);
    const void* d = exact(a[2], at::kFloat, {x.rows, K}, dev);
    const int64_t score = integer(a[3]);
    const int renormalize = PyObject_IsTrue(a[4]);
    need(renormalize >= 0);
    void* stream = stream_on(a[5], a[6], dev);
    const at::Tensor out = at::empty({x.rows, x.cols}, x.t.options());
    const int status = unlocked([&] {
      return g_route_backward(x.t.data_ptr(), x.dtype, x.rows, (int32_t)x.cols, x.ld, ints(ids),
                              static_cast<const float*>(d), (int32_t)K, (int)score, renormalize, out.data_ptr(),
                              x.cols, stream);
    });
    need(status == MOE_FP4_OK);
    return THPVariable_Wrap(out);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef kMethods[] = {
    {"quantize_fp8", method<quantize_fp8>(), METH_FASTCALL, nullptr},
    {"gemm_fp8", method<gemm_fp8>(), METH_FASTCALL, nullptr},
    {"dispatch", method<dispatch>(), METH_FASTCALL, nullptr},
    {"dispatch_backward", method<dispatch_backward>(), METH_FASTCALL, nullptr},
    {"combine_backward", method<combine_backward>(), METH_FASTCALL, nullptr},
    {"route_backward", method<route_backward>(), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"ffn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ffn)), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&kModule); }
