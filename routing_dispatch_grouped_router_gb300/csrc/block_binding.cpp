// Python module _block: the operators around the layer on torch tensors.
//
// It checks shapes, types, strides and devices, makes the outputs and scratch
// that the caller gave none for, and calls the C ABI (include/mok.h); it
// computes nothing.  A decode step makes several of these calls one after the
// other, so their host time counts: one call of the same checks and allocations
// in Python took 12 to 28 us on a Grace core, three times the kernel's.
//
// Every tensor made here is allocated on the stream that the call runs on (the
// current one or the given one), so that its memory is not handed out again
// before that stream is done with it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "../../include/mok.h"

namespace {

PyObject* g_raise = nullptr;   // raise(code, where): the package's error of a status code
PyObject* g_status = nullptr;  // status(device index): address of the device status word
int64_t g_status_addr[64] = {0};

struct MokFail {
  int code;
  const char* where;
};

void check(mok_status s, const char* where) {
  if (s != MOK_OK) throw MokFail{static_cast<int>(s), where};
}

template <typename F>
PyObject* guarded(const F& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const MokFail& e) {
    PyObject* r = PyObject_CallFunction(g_raise, "is", e.code, e.where);
    Py_XDECREF(r);  // (it raises)
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.where);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

const at::Tensor* tensor_or_null(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_null(o, name);
  TORCH_CHECK_VALUE(t != nullptr, name, " is needed");
  return *t;
}
void* addr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* addr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
// (a tensor of several elements, for one, has no truth value)
bool flag(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) PyErr_Clear();
  TORCH_CHECK_VALUE(v >= 0, name, " must be true or false");
  return v != 0;
}

// The stream of a call on the GPU of `t`, which must be the current one.
struct Call {
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  cudaStream_t raw = nullptr;
  c10::Device device;
  Call(const at::Tensor& t, PyObject* stream) : device(t.device()) {
    TORCH_CHECK_VALUE(t.is_cuda() && device.index() == c10::cuda::current_device(),
                      "the tensors must be on the current GPU, not on ", device.str());
    if (stream == Py_None) {
      raw = c10::cuda::getCurrentCUDAStream(device.index()).stream();
      return;
    }
    int64_t v[3];
    const char* names[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
      PyObject* a = PyObject_GetAttrString(stream, names[i]);
      if (!a) throw python_error();
      v[i] = PyLong_AsLongLong(a);
      Py_DECREF(a);
    }
    const auto s = c10::cuda::CUDAStream::unpack3(
        v[0], static_cast<c10::DeviceIndex>(v[1]), static_cast<c10::DeviceType>(v[2]));
    TORCH_CHECK_VALUE(s.device_index() == device.index(),
                      "the stream must be of the tensors' GPU");
    guard.emplace(s);
    raw = s.stream();
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dt) const {
    return at::Tensor(at::detail::empty_cuda(shape, dt, device, std::nullopt));
  }
  int32_t* status() const {
    const int i = device.index();
    TORCH_CHECK(i < 64, "device index");
    if (g_status_addr[i] == 0) {
      PyObject* r = PyObject_CallFunction(g_status, "i", i);
      if (!r) throw python_error();
      g_status_addr[i] = PyLong_AsLongLong(r);
      Py_DECREF(r);
    }
    return reinterpret_cast<int32_t*>(g_status_addr[i]);
  }
};

bool real(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
int elem(at::ScalarType t) { return t == at::kFloat ? MOK_ELEM_F32 : MOK_ELEM_BF16; }

void same_device(const at::Tensor& t, const char* name, c10::Device d) {
  TORCH_CHECK_VALUE(t.device() == d, name, " must be on the GPU of the other tensors, not on ",
                    t.device().str());
}

// A matrix with consecutive columns: its row stride.
int64_t matrix(const at::Tensor& t, const char* name, c10::Device d) {
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must be a matrix");
  same_device(t, name, d);
  const int64_t rows = t.size(0), cols = t.size(1);
  TORCH_CHECK_VALUE(cols <= 1 || t.stride(1) == 1, name, " must have consecutive columns");
  if (rows <= 1) return cols;
  TORCH_CHECK_VALUE(t.stride(0) >= cols, name, " must have rows that do not overlap");
  return t.stride(0);
}
int64_t matrix(const at::Tensor& t, const char* name, c10::Device d, int64_t rows, int64_t cols) {
  const int64_t ld = matrix(t, name, d);
  TORCH_CHECK_VALUE(t.size(0) == rows && t.size(1) == cols, name, " must be [", rows, ", ", cols,
                    "], got ", t.sizes());
  return ld;
}
void type_is(const at::Tensor& t, const char* name, at::ScalarType a) {
  TORCH_CHECK_VALUE(t.scalar_type() == a, name, " must not be ", t.scalar_type());
}
void type_real(const at::Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(real(t.scalar_type()), name, " must not be ", t.scalar_type());
}
void dense(const at::Tensor& t, const char* name, c10::Device d, at::IntArrayRef shape) {
  same_device(t, name, d);
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must be ", shape, ", got ", t.sizes());
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o;
    if (t.defined()) {
      o = wrap(t);
    } else {
      Py_INCREF(Py_None);
      o = Py_None;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Scratch: the caller's, or made here (freed on this stream when the call returns).
struct Scratch {
  at::Tensor own;
  void* p;
  size_t n;
  Scratch(const Call& c, const at::Tensor* given, size_t bytes) {
    if (given) {
      same_device(*given, "workspace", c.device);
      TORCH_CHECK_VALUE(given->is_contiguous(), "workspace must be contiguous");
      p = given->data_ptr();
      n = given->nbytes();
    } else {
      p = nullptr;
      n = bytes;
      if (bytes == 0) return;
      own = c.empty({static_cast<int64_t>(bytes)}, at::kByte);
      p = own.data_ptr();
    }
  }
};

// ------------------------------------------------------------- add_rmsnorm --

mok_rmsnorm_desc norm_desc(const Call& c, const at::Tensor& x, const at::Tensor& weight,
                           const at::Tensor* res, at::Tensor& s, double eps) {
  mok_rmsnorm_desc D = {};
  D.ld_x = matrix(x, "x", c.device);
  type_real(x, "x");
  D.rows = x.size(0);
  D.d = x.size(1);
  dense(weight, "weight", c.device, {D.d});
  type_real(weight, "weight");
  D.eps = static_cast<float>(eps);
  const at::ScalarType st = res ? res->scalar_type() : x.scalar_type();
  if (res) {
    D.ld_res = matrix(*res, "residual", c.device, D.rows, D.d);
    type_real(*res, "residual");
    if (!s.defined()) s = c.empty({D.rows, D.d}, st);
  }
  if (s.defined()) {
    D.ld_s = matrix(s, "s", c.device, D.rows, D.d);
    type_is(s, "s", st);
  }
  D.x_elem = elem(x.scalar_type());
  D.s_elem = elem(st);
  D.weight_elem = elem(weight.scalar_type());
  return D;
}

// (x, weight, residual, eps, s, y, stream) -> (s, y)
PyObject* py_add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor& w = tensor(a[1], "weight");
    const at::Tensor* res = tensor_or_null(a[2], "residual");
    const at::Tensor *s0 = tensor_or_null(a[4], "s"), *y0 = tensor_or_null(a[5], "y");
    const Call c(x, a[6]);
    at::Tensor s = s0 ? *s0 : at::Tensor();
    mok_rmsnorm_desc D = norm_desc(c, x, w, res, s, number(a[3]));
    at::Tensor y = y0 ? *y0 : c.empty({D.rows, D.d}, at::kBFloat16);
    D.ld_y = matrix(y, "y", c.device, D.rows, D.d);
    type_is(y, "y", at::kBFloat16);
    check(mok_add_rmsnorm_forward(&D, addr(x), addr(res), addr(w), addr(s), addr(y), nullptr,
                                  nullptr, nullptr, c.raw),
          "mok_add_rmsnorm_forward");
    return tuple({s.defined() ? s : x, y});
  });
}

// (x, weight, residual, eps, s, y, values, codes, scales, stream) -> (s, codes, scales)
PyObject* py_add_rmsnorm_mx(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor& w = tensor(a[1], "weight");
    const at::Tensor* res = tensor_or_null(a[2], "residual");
    const at::Tensor *s0 = tensor_or_null(a[4], "s"), *y = tensor_or_null(a[5], "y");
    const at::Tensor *values = tensor_or_null(a[6], "values"), *c0 = tensor_or_null(a[7], "codes"),
                     *e0 = tensor_or_null(a[8], "scales");
    const Call c(x, a[9]);
    at::Tensor s = s0 ? *s0 : at::Tensor();
    mok_rmsnorm_desc D = norm_desc(c, x, w, res, s, number(a[3]));
    TORCH_CHECK_VALUE(D.d % 32 == 0, "MXFP8 needs d a multiple of 32");
    at::Tensor codes = c0 ? *c0 : c.empty({D.rows, D.d}, at::kByte);
    at::Tensor scales = e0 ? *e0 : c.empty({D.rows, D.d / 32}, at::kByte);
    dense(codes, "codes", c.device, {D.rows, D.d});
    type_is(codes, "codes", at::kByte);
    dense(scales, "scales", c.device, {D.rows, D.d / 32});
    type_is(scales, "scales", at::kByte);
    if (y) {
      D.ld_y = matrix(*y, "y", c.device, D.rows, D.d);
      type_is(*y, "y", at::kBFloat16);
    }
    if (values) {
      dense(*values, "values", c.device, {D.rows, D.d});
      type_is(*values, "values", at::kBFloat16);
    }
    check(mok_add_rmsnorm_forward(&D, addr(x), addr(res), addr(w), addr(s), addr(y), addr(values),
                                  static_cast<uint8_t*>(addr(codes)),
                                  static_cast<uint8_t*>(addr(scales)), c.raw),
          "mok_add_rmsnorm_forward");
    return tuple({s.defined() ? s : x, codes, scales});
  });
}

// (dy, s, weight, ds, eps, dx, dweight, accumulate, workspace, stream) -> (dx, dweight)
PyObject* py_add_rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor& dy = tensor(a[0], "dy");
    const at::Tensor& s = tensor(a[1], "s");
    const at::Tensor& w = tensor(a[2], "weight");
    const at::Tensor* ds = tensor_or_null(a[3], "ds");
    const at::Tensor *dx0 = tensor_or_null(a[5], "dx"), *dw0 = tensor_or_null(a[6], "dweight");
    const bool acc = flag(a[7], "accumulate");
    const Call c(dy, a[9]);
    mok_rmsnorm_desc D = {};
    D.ld_x = matrix(dy, "dy", c.device);
    type_real(dy, "dy");
    D.rows = dy.size(0);
    D.d = dy.size(1);
    D.ld_s = matrix(s, "s", c.device, D.rows, D.d);
    type_real(s, "s");
    dense(w, "weight", c.device, {D.d});
    type_real(w, "weight");
    if (ds) {
      D.ld_res = matrix(*ds, "ds", c.device, D.rows, D.d);
      type_is(*ds, "ds", s.scalar_type());
    }
    TORCH_CHECK_VALUE(dw0 || !acc, "accumulate needs dweight");
    at::Tensor dx = dx0 ? *dx0 : c.empty({D.rows, D.d}, s.scalar_type());
    D.ld_y = matrix(dx, "dx", c.device, D.rows, D.d);
    type_is(dx, "dx", s.scalar_type());
    at::Tensor dw = dw0 ? *dw0 : c.empty({D.d}, at::kFloat);
    dense(dw, "dweight", c.device, {D.d});
    type_is(dw, "dweight", at::kFloat);
    D.eps = static_cast<float>(number(a[4]));
    D.x_elem = elem(dy.scalar_type());
    D.s_elem = elem(s.scalar_type());
    D.weight_elem = elem(w.scalar_type());
    D.accumulate = acc;
    size_t n = 0;
    check(mok_add_rmsnorm_workspace_size(&D, &n), "mok_add_rmsnorm_workspace_size");
    const Scratch ws(c, tensor_or_null(a[8], "workspace"), n);
    check(mok_add_rmsnorm_backward(&D, addr(dy), addr(s), addr(w), addr(ds), addr(dx),
                                   static_cast<float*>(addr(dw)), ws.p, ws.n, c.status(), c.raw),
          "mok_add_rmsnorm_backward");
    return tuple({dx, dw});
  });
}

// ---------------------------------------------------------- router_balance --

mok_balance_desc balance_desc(const Call& c, const at::Tensor& logits, int64_t k,
                              const at::Tensor* mask, double balance_coef, double z_coef) {
  mok_balance_desc D = {};
  D.ld_logits = matrix(logits, "logits", c.device);
  type_is(logits, "logits", at::kFloat);
  D.T = logits.size(0);
  TORCH_CHECK_VALUE(logits.size(1) < (1LL << 31) && k < (1LL << 31), "E and k are 32-bit");
  D.E = static_cast<int32_t>(logits.size(1));
  D.k = static_cast<int32_t>(k);
  if (mask) {
    dense(*mask, "mask", c.device, {D.T});
    TORCH_CHECK_VALUE(mask->scalar_type() == at::kByte || mask->scalar_type() == at::kBool,
                      "mask must not be ", mask->scalar_type());
  }
  D.balance_coef = static_cast<float>(balance_coef);
  D.z_coef = static_cast<float>(z_coef);
  return D;
}

// (logits, topk_idx, mask, balance_coef, z_coef, workspace, stream) ->
//   (loss, counts, prob, lse, n_valid)
PyObject* py_router_balance(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor& logits = tensor(a[0], "logits");
    const at::Tensor& idx = tensor(a[1], "topk_idx");
    const at::Tensor* mask = tensor_or_null(a[2], "mask");
    const Call c(logits, a[6]);
    TORCH_CHECK_VALUE(idx.dim() == 2, "topk_idx must be a matrix");
    const mok_balance_desc D =
        balance_desc(c, logits, idx.size(1), mask, number(a[3]), number(a[4]));
    dense(idx, "topk_idx", c.device, {D.T, D.k});
    type_is(idx, "topk_idx", at::kInt);
    at::Tensor loss = c.empty({2}, at::kFloat), counts = c.empty({D.E}, at::kInt),
               prob = c.empty({D.E}, at::kFloat), lse = c.empty({D.T}, at::kFloat),
               nv = c.empty({1}, at::kInt);
    size_t n = 0;
    check(mok_router_balance_workspace_size(&D, &n), "mok_router_balance_workspace_size");
    const Scratch ws(c, tensor_or_null(a[5], "workspace"), n);
    check(mok_router_balance_forward(
              &D, static_cast<float*>(addr(logits)), static_cast<int32_t*>(addr(idx)),
              static_cast<uint8_t*>(addr(mask)), static_cast<float*>(addr(loss)),
              static_cast<int32_t*>(addr(counts)), static_cast<float*>(addr(prob)),
              static_cast<float*>(addr(lse)), static_cast<int32_t*>(addr(nv)), ws.p, ws.n,
              c.status(), c.raw),
          "mok_router_balance_forward");
    return tuple({loss, counts, prob, lse, nv});
  });
}

// (dloss, logits, lse, counts, n_valid, k, mask, balance_coef, z_coef, dlogits, stream) -> dlogits
PyObject* py_router_balance_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor& dloss = tensor(a[0], "dloss");
    const at::Tensor& logits = tensor(a[1], "logits");
    const at::Tensor& lse = tensor(a[2], "lse");
    const at::Tensor& counts = tensor(a[3], "counts");
    const at::Tensor& nv = tensor(a[4], "n_valid");
    const at::Tensor* mask = tensor_or_null(a[6], "mask");
    const at::Tensor* dl0 = tensor_or_null(a[9], "dlogits");
    const Call c(logits, a[10]);
    const mok_balance_desc D =
        balance_desc(c, logits, integer(a[5]), mask, number(a[7]), number(a[8]));
    dense(dloss, "dloss", c.device, {2});
    type_is(dloss, "dloss", at::kFloat);
    dense(lse, "lse", c.device, {D.T});
    type_is(lse, "lse", at::kFloat);
    dense(counts, "counts", c.device, {D.E});
    type_is(counts, "counts", at::kInt);
    dense(nv, "n_valid", c.device, {1});
    type_is(nv, "n_valid", at::kInt);
    at::Tensor dl;
    if (dl0) {
      dl = *dl0;
    } else {
      dl = c.empty({D.T, D.ld_logits}, at::kFloat);
      if (D.ld_logits != D.E) dl = dl.narrow(1, 0, D.E);
    }
    type_is(dl, "dlogits", at::kFloat);
    TORCH_CHECK_VALUE(matrix(dl, "dlogits", c.device, D.T, D.E) == D.ld_logits,
                      "dlogits must have the row stride of logits");
    check(mok_router_balance_backward(
              &D, static_cast<float*>(addr(dloss)), static_cast<float*>(addr(logits)),
              static_cast<float*>(addr(lse)), static_cast<int32_t*>(addr(counts)),
              static_cast<int32_t*>(addr(nv)), static_cast<uint8_t*>(addr(mask)),
              static_cast<float*>(addr(dl)), c.raw),
          "mok_router_balance_backward");
    return wrap(dl);
  });
}

// ----------------------------------------------------------------- linear --

at::ScalarType dtype_or(PyObject* o, at::ScalarType other, const char* name) {
  if (o == Py_None) return other;
  TORCH_CHECK_VALUE(THPDtype_Check(o), name, " must be a torch.dtype");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  TORCH_CHECK_VALUE(real(t), name, " must not be ", t);
  return t;
}

// x [M, K], w [N, K]: sizes, x's stride and the activation
mok_linear_desc linear_desc(const Call& c, const at::Tensor& x, const at::Tensor& w, int64_t act) {
  mok_linear_desc D = {};
  D.ld_x = matrix(x, "x", c.device);
  type_is(x, "x", at::kBFloat16);
  D.M = x.size(0);
  D.K = x.size(1);
  TORCH_CHECK_VALUE(w.dim() == 2, "w must be a matrix");
  D.N = w.size(0);
  dense(w, "w", c.device, {D.N, D.K});
  type_is(w, "w", at::kBFloat16);
  D.act = static_cast<int32_t>(act);
  return D;
}

// (x, w, bias, act, residual, out_dtype, y, z, keep_z, workspace, stream) -> y or (y, z)
PyObject* py_linear(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor& w = tensor(a[1], "w");
    const at::Tensor* bias = tensor_or_null(a[2], "bias");
    const at::Tensor* res = tensor_or_null(a[4], "residual");
    const at::Tensor *y0 = tensor_or_null(a[6], "y"), *z0 = tensor_or_null(a[7], "z");
    const bool keep = flag(a[8], "keep_z");
    const Call c(x, a[10]);
    mok_linear_desc D = linear_desc(c, x, w, integer(a[3]));
    const at::ScalarType dt =
        dtype_or(a[5], y0 ? y0->scalar_type() : at::kBFloat16, "out_dtype");
    TORCH_CHECK_VALUE(real(dt), "y must not be ", dt);
    if (bias) {
      dense(*bias, "bias", c.device, {D.N});
      type_is(*bias, "bias", at::kFloat);
    }
    at::Tensor y = y0 ? *y0 : c.empty({D.M, D.N}, dt);
    at::Tensor z = z0 ? *z0 : (keep ? c.empty({D.M, D.N}, dt) : at::Tensor());
    dense(y, "y", c.device, {D.M, D.N});
    type_is(y, "y", dt);
    if (z.defined()) {
      dense(z, "z", c.device, {D.M, D.N});
      type_is(z, "z", dt);
    }
    if (res) {
      dense(*res, "residual", c.device, {D.M, D.N});
      type_is(*res, "residual", dt);
    }
    D.y_elem = elem(dt);
    size_t n = 0;
    check(mok_linear_workspace_size(&D, 0, &n), "mok_linear_workspace_size");
    const Scratch ws(c, tensor_or_null(a[9], "workspace"), n);
    check(mok_linear_forward(&D, addr(x), addr(w), static_cast<float*>(addr(bias)), addr(res),
                             addr(y), addr(z), ws.p, ws.n, c.status(), c.raw),
          "mok_linear_forward");
    return keep ? tuple({y, z}) : wrap(y);
  });
}

// (dy, x, w, z, act, bias, dx_dtype, dx, dw, dbias, accumulate, workspace, stream) ->
//   (dx, dw, dbias)
PyObject* py_linear_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor& dy = tensor(a[0], "dy");
    const at::Tensor& x = tensor(a[1], "x");
    const at::Tensor& w = tensor(a[2], "w");
    const int64_t act = integer(a[4]);
    const at::Tensor* z = act == MOK_ACT_NONE ? nullptr : tensor_or_null(a[3], "z");
    const at::Tensor *dx0 = tensor_or_null(a[7], "dx"), *dw0 = tensor_or_null(a[8], "dw"),
                     *db0 = tensor_or_null(a[9], "dbias");
    const bool bias = flag(a[5], "bias") || db0 != nullptr;
    const int64_t acc = integer(a[10]);
    const Call c(x, a[12]);
    mok_linear_desc D = linear_desc(c, x, w, act);
    dense(dy, "dy", c.device, {D.M, D.N});
    type_real(dy, "dy");
    TORCH_CHECK_VALUE(act == MOK_ACT_NONE || z, "the activation's gradient needs z");
    if (z) {
      dense(*z, "z", c.device, {D.M, D.N});
      type_is(*z, "z", dy.scalar_type());
    }
    TORCH_CHECK_VALUE(!(acc & MOK_ADD_DX) || dx0, "accumulate needs dx to add into");
    TORCH_CHECK_VALUE(!(acc & MOK_ADD_DW) || (dw0 && (!bias || db0)),
                      "accumulate needs dw and dbias to add into");
    const at::ScalarType dt =
        dtype_or(a[6], dx0 ? dx0->scalar_type() : at::kBFloat16, "dx_dtype");
    TORCH_CHECK_VALUE(real(dt), "dx must not be ", dt);
    at::Tensor dx = dx0 ? *dx0 : c.empty({D.M, D.K}, dt);
    at::Tensor dw = dw0 ? *dw0 : c.empty({D.N, D.K}, at::kFloat);
    at::Tensor db = db0 ? *db0 : (bias ? c.empty({D.N}, at::kFloat) : at::Tensor());
    dense(dx, "dx", c.device, {D.M, D.K});
    type_is(dx, "dx", dt);
    dense(dw, "dw", c.device, {D.N, D.K});
    type_is(dw, "dw", at::kFloat);
    if (bias) {
      dense(db, "dbias", c.device, {D.N});
      type_is(db, "dbias", at::kFloat);
    }
    D.y_elem = elem(dy.scalar_type());
    D.dx_elem = elem(dt);
    D.accumulate = static_cast<int32_t>(acc);
    size_t n = 0;
    const bool aligned = (reinterpret_cast<uintptr_t>(addr(dy)) & 15) == 0;
    check(mok_linear_workspace_size(&D, aligned ? 2 : 1, &n), "mok_linear_workspace_size");
    const Scratch ws(c, tensor_or_null(a[11], "workspace"), n);
    check(mok_linear_backward(&D, addr(dy), addr(x), addr(w), addr(z), addr(dx),
                              static_cast<float*>(addr(dw)), static_cast<float*>(addr(db)), ws.p,
                              ws.n, c.status(), c.raw),
          "mok_linear_backward");
    return tuple({dx, dw, db});
  });
}

// (raise, status): the two callables above
PyObject* py_setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "setup(raise, status)");
    return nullptr;
  }
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  g_raise = a[0];
  g_status = a[1];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
    return nullptr;
  }
  return F(self, a, n);
}

#define MOK_METHOD(name, n)                                                              \
  {#name, reinterpret_cast<PyCFunction>(                                                 \
              reinterpret_cast<void (*)()>(&counted<py_##name, n>)),                     \
   METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    MOK_METHOD(setup, 2),
    MOK_METHOD(add_rmsnorm, 7),
    MOK_METHOD(add_rmsnorm_mx, 10),
    MOK_METHOD(add_rmsnorm_backward, 10),
    MOK_METHOD(router_balance, 7),
    MOK_METHOD(router_balance_backward, 11),
    MOK_METHOD(linear, 11),
    MOK_METHOD(linear_backward, 13),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
