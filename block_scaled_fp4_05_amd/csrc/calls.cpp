// Short host path of the Python binding's few-token calls (a CPython extension module;
// no device code).
//
// These calls run a few microseconds on the GPU, and checking a dozen tensors and
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
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind: five addresses");
    return nullptr;
  }
  uintptr_t p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = (uintptr_t)PyLong_AsUnsignedLongLong(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
  g_ffn = reinterpret_cast<decltype(g_ffn)>(p[1]);
  g_ffn_workspace = reinterpret_cast<decltype(g_ffn_workspace)>(p[2]);
  g_route = reinterpret_cast<decltype(g_route)>(p[3]);
  g_route_workspace = reinterpret_cast<decltype(g_route_workspace)>(p[4]);
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

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"ffn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ffn)), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&kModule); }
