// Python binding of the layer operators: checks of torch tensors, allocation of the
// outputs that the caller does not pass, and the C calls of include/phobos_layers.h.
//
// A product or norm of one token takes 4 to 9 us on the GPU; the same checks in Python
// took 12 us a call.  layers.py documents and names the arguments and passes them by
// position; the entry points arrive as addresses (bind), so that this module and the
// library do not depend on each other to load.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <new>

#include "../../include/phobos_layers.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Entries {
  phobos_status_t (*linear)(const phobos_linear_args_t *, void *);
  phobos_status_t (*linear_backward)(const phobos_linear_backward_args_t *, void *);
  phobos_status_t (*rmsnorm)(const phobos_rmsnorm_args_t *, void *);
  phobos_status_t (*rmsnorm_backward)(const phobos_rmsnorm_backward_args_t *, void *);
} entries = {};

// A Python exception is set; unwinds to the module function.
struct Raised {};
template <typename... Args>
[[noreturn]] void raise(PyObject *type, const char *format, Args... args) {
  PyErr_Format(type, format, args...);
  throw Raised();
}

long long ll(int64_t x) { return static_cast<long long>(x); }

// ------------------------------------------------------------------- arguments

// Autograd does not see these calls, so what it would record is refused rather than lost.
const Tensor *optional_tensor(PyObject *o, const char *name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  const Tensor &t = THPVariable_Unpack(o);
  if (t.requires_grad() && c10::GradMode::is_enabled())
    raise(PyExc_ValueError,
          "%s requires grad, which the layer operators do not record: call them under torch.no_grad() (as inside "
          "a torch.autograd.Function), or detach it",
          name);
  return &t;
}

const Tensor &tensor(PyObject *o, const char *name) {
  const Tensor *t = optional_tensor(o, name);
  if (!t) raise(PyExc_TypeError, "%s must be a tensor", name);
  return *t;
}

int64_t integer(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

ScalarType dtype_or(PyObject *o, ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, "a dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// The library's code of a floating type, or -1.
int float_type(ScalarType t) {
  return t == ScalarType::Float      ? PHOBOS_TYPE_F32
         : t == ScalarType::Half     ? PHOBOS_TYPE_F16
         : t == ScalarType::BFloat16 ? PHOBOS_TYPE_BF16
                                     : -1;
}

int need_float_type(ScalarType t, const char *name) {
  const int code = float_type(t);
  if (code < 0) raise(PyExc_TypeError, "%s has unsupported dtype %s", name, c10::toString(t));
  return code;
}

void need_2d(const Tensor &t, const char *name) {
  if (!t.is_cuda()) raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
  if (t.dim() != 2) raise(PyExc_ValueError, "%s must be 2-D", name);
}

void need_kind(const Tensor &t, const char *name, ScalarType type, c10::DeviceIndex index) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != index)
    raise(PyExc_TypeError, "%s must be a %s tensor on cuda:%d", name, c10::toString(type), static_cast<int>(index));
}

void need_shape(const Tensor &t, const char *name, int64_t rows, int64_t cols) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    raise(PyExc_ValueError, "%s must have shape (%lld, %lld)", name, ll(rows), ll(cols));
}

// The row stride of a row-major matrix with unit inner stride.
int64_t row_stride(const Tensor &t, const char *name, int64_t rows, int64_t cols, ScalarType type,
                   c10::DeviceIndex index) {
  need_kind(t, name, type, index);
  need_shape(t, name, rows, cols);
  const int64_t row = t.stride(0), col = t.stride(1);
  if ((cols > 1 && rows > 0 && col != 1) || (rows > 1 && row < cols))
    raise(PyExc_ValueError, "%s must be row-major with unit inner stride", name);
  return rows > 1 ? row : std::max<int64_t>(cols, 1);
}

void *vector(const Tensor &t, const char *name, int64_t n, ScalarType type, c10::DeviceIndex index) {
  need_kind(t, name, type, index);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    raise(PyExc_ValueError, "%s must be a contiguous vector of %lld", name, ll(n));
  return t.data_ptr();
}

struct Strides {
  int64_t row, col;
};

// The strides of a matrix with a unit stride in either dimension; those that no
// element depends on are filled in.
Strides strided(const Tensor &t, const char *name) {
  const int64_t rows = t.size(0), cols = t.size(1), row = t.stride(0), col = t.stride(1);
  if (rows == 0 || cols == 0) return {std::max<int64_t>(cols, 1), 1};
  if (cols == 1) return {rows > 1 ? row : 1, 1};
  if (rows == 1) return col == 1 ? Strides{cols, 1} : Strides{1, col};
  if (col == 1 && row >= cols) return {row, 1};
  if (row != 1 || col < rows)
    raise(PyExc_ValueError, "%s must have a unit stride and no overlapping rows", name);
  return {1, col};
}

Tensor new_matrix(int64_t rows, int64_t cols, ScalarType type, const Tensor &like) {
  return at::empty({rows, cols}, at::TensorOptions().dtype(type).device(like.device()));
}

// ------------------------------------------------------------------------ calls

template <typename Entry, typename Args>
PyObject *status(Entry entry, const Args &args, c10::DeviceIndex index) {
  if (!entry) raise(PyExc_RuntimeError, "the library is not bound");
  void *stream = c10::cuda::getCurrentCUDAStream(index).stream();
  phobos_status_t st;
  Py_BEGIN_ALLOW_THREADS st = entry(&args, stream);
  Py_END_ALLOW_THREADS return st == PHOBOS_OK ? nullptr : PyLong_FromLong(st);
}

PyObject *wrap(const Tensor *t) {
  if (!t || !t->defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}

// A non-zero status as an int, or else the tuple of results.
template <size_t N>
PyObject *results(PyObject *failed, const Tensor *const (&tensors)[N]) {
  if (failed) return failed;
  PyObject *tuple = PyTuple_New(N);
  if (!tuple) throw Raised();
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(tuple, i, wrap(tensors[i]));
  return tuple;
}

// Tells autograd that a tensor of the caller's has changed: one that was saved for a
// backward pass is then found to have.
void written(const Tensor *t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// x, w, x_scale, w_scale, bias, residual, act, out, out_dtype, preact, save_preact, products
PyObject *linear(PyObject *const *a) {
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
  const Tensor *x_scale = optional_tensor(a[2], "x_scale"), *w_scale = optional_tensor(a[3], "w_scale");
  const Tensor *bias = optional_tensor(a[4], "bias"), *residual = optional_tensor(a[5], "residual");
  const Tensor *given_out = optional_tensor(a[7], "out"), *given_preact = optional_tensor(a[9], "preact");
  if (given_out && dtype_or(a[8], given_out->scalar_type()) != given_out->scalar_type())
    raise(PyExc_TypeError, "out is a %s tensor, not out_dtype", c10::toString(given_out->scalar_type()));
  need_2d(x, "x");
  need_2d(w, "w");
  const c10::DeviceIndex index = x.get_device();
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  const ScalarType type = x.scalar_type();
  need_kind(w, "w", type, index);
  phobos_linear_args_t p = {};
  p.M = x.size(0);
  p.K = x.size(1);
  p.N = w.size(1);
  if (w.size(0) != p.K)
    raise(PyExc_ValueError, "shape mismatch: x (%lld, %lld), w (%lld, %lld)", ll(p.M), ll(p.K), ll(w.size(0)), ll(p.N));
  const Strides xs = strided(x, "x"), ws = strided(w, "w");
  if (x_scale || w_scale) {
    if (!x_scale || !w_scale) raise(PyExc_TypeError, "8-bit operands need x_scale and w_scale");
    if (type != ScalarType::Float8_e4m3fn) raise(PyExc_TypeError, "x has unsupported dtype %s", c10::toString(type));
    if (p.K > 1 && (xs.col != 1 || ws.row != 1))
      raise(PyExc_ValueError,
            "8-bit operands need unit stride along K: x row-major, w the transposed view of an N x K tensor");
    p.type = PHOBOS_TYPE_E4M3;
    p.x_scale = static_cast<const float *>(vector(*x_scale, "x_scale", p.M, ScalarType::Float, index));
    p.w_scale = static_cast<const float *>(vector(*w_scale, "w_scale", p.N, ScalarType::Float, index));
  } else {
    p.type = need_float_type(type, "x");
  }
  const ScalarType out_type = given_out ? given_out->scalar_type() : dtype_or(a[8], type);
  p.out_type = need_float_type(out_type, "out");
  p.act = static_cast<int32_t>(integer(a[6]));
  p.products = static_cast<int32_t>(integer(a[11]));
  Tensor out, preact;
  if (given_out) p.out_row = row_stride(*given_out, "out", p.M, p.N, out_type, index);
  if (given_preact) p.preact_row = row_stride(*given_preact, "preact", p.M, p.N, out_type, index);
  if (residual) {
    p.residual_row = row_stride(*residual, "residual", p.M, p.N, out_type, index);
    p.residual = residual->data_ptr();
  }
  if (bias) p.bias = vector(*bias, "bias", p.N, out_type, index);
  if (!given_out) {
    out = new_matrix(p.M, p.N, out_type, x);
    p.out_row = std::max<int64_t>(p.N, 1);
    given_out = &out;
  }
  if (!given_preact && truth(a[10])) {
    preact = new_matrix(p.M, p.N, out_type, x);
    p.preact_row = std::max<int64_t>(p.N, 1);
    given_preact = &preact;
  }
  p.x = x.data_ptr();
  p.x_row = xs.row;
  p.x_col = xs.col;
  p.w = w.data_ptr();
  p.w_row = ws.row;
  p.w_col = ws.col;
  p.out = given_out->data_ptr();
  if (given_preact) p.preact = given_preact->data_ptr();
  for (const Tensor *t : {given_out, given_preact}) written(t);
  return results(status(entries.linear, p, index), {given_out, given_preact});
}

// dout, x, w, preact, act, dx, dw, dbias, need_dx, need_dw, need_dbias, grad_dtype, accumulate, products
PyObject *linear_backward(PyObject *const *a) {
  const Tensor &dout = tensor(a[0], "dout"), &x = tensor(a[1], "x"), &w = tensor(a[2], "w");
  const Tensor *preact = optional_tensor(a[3], "preact");
  const bool need_dx = truth(a[8]), need_dw = truth(a[9]), need_dbias = truth(a[10]);
  const Tensor *dx = need_dx ? optional_tensor(a[5], "dx") : nullptr;
  const Tensor *dw = need_dw ? optional_tensor(a[6], "dw") : nullptr;
  const Tensor *dbias = need_dbias ? optional_tensor(a[7], "dbias") : nullptr;
  need_2d(x, "x");
  need_2d(w, "w");
  const c10::DeviceIndex index = x.get_device();
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  const ScalarType type = x.scalar_type();
  need_kind(w, "w", type, index);
  phobos_linear_backward_args_t p = {};
  p.type = need_float_type(type, "x");
  p.M = x.size(0);
  p.K = x.size(1);
  p.N = w.size(1);
  if (w.size(0) != p.K)
    raise(PyExc_ValueError, "shape mismatch: x (%lld, %lld), w (%lld, %lld)", ll(p.M), ll(p.K), ll(w.size(0)), ll(p.N));
  p.act = static_cast<int32_t>(integer(a[4]));
  p.accumulate = truth(a[12]);
  p.products = static_cast<int32_t>(integer(a[13]));
  if (p.act != PHOBOS_ACT_NONE && !preact) raise(PyExc_ValueError, "the gradient of an activation needs preact");
  if (p.accumulate && ((need_dw && !dw) || (need_dbias && !dbias)))
    raise(PyExc_ValueError, "accumulate needs the tensors to add to");
  p.dout_row = row_stride(dout, "dout", p.M, p.N, type, index);
  p.dout = dout.data_ptr();
  const Strides xs = strided(x, "x"), ws = strided(w, "w");
  if (p.act != PHOBOS_ACT_NONE) {
    p.preact_row = row_stride(*preact, "preact", p.M, p.N, type, index);
    p.preact = preact->data_ptr();
  }
  const ScalarType grad_type = dtype_or(a[11], dw ? dw->scalar_type() : dbias ? dbias->scalar_type() : type);
  if (grad_type != type && grad_type != ScalarType::Float)
    raise(PyExc_TypeError, "gradients of %s weights are %s or float32", c10::toString(type), c10::toString(type));
  p.grad_type = float_type(grad_type);
  Strides dws = {1, 1};
  if (dx) p.dx_row = row_stride(*dx, "dx", p.M, p.K, type, index);
  if (dw) {
    need_kind(*dw, "dw", grad_type, index);
    need_shape(*dw, "dw", p.K, p.N);
    dws = strided(*dw, "dw");
  }
  if (dbias) vector(*dbias, "dbias", p.N, grad_type, index);
  Tensor new_dx, new_dw, new_dbias;
  if (need_dx && !dx) {
    new_dx = new_matrix(p.M, p.K, type, x);
    p.dx_row = std::max<int64_t>(p.K, 1);
    dx = &new_dx;
  }
  if (need_dw && !dw) {  // in w's layout
    new_dw = ws.col == 1 ? new_matrix(p.K, p.N, grad_type, x) : new_matrix(p.N, p.K, grad_type, x).t();
    dws = strided(new_dw, "dw");
    dw = &new_dw;
  }
  if (need_dbias && !dbias) {
    new_dbias = at::empty({p.N}, at::TensorOptions().dtype(grad_type).device(x.device()));
    dbias = &new_dbias;
  }
  p.x = x.data_ptr();
  p.x_row = xs.row;
  p.x_col = xs.col;
  p.w = w.data_ptr();
  p.w_row = ws.row;
  p.w_col = ws.col;
  if (dx) p.dx = dx->data_ptr();
  if (dw) p.dw = dw->data_ptr();
  p.dw_row = dws.row;
  p.dw_col = dws.col;
  if (dbias) p.dbias = dbias->data_ptr();
  for (const Tensor *t : {dx, dw, dbias}) written(t);
  return results(status(entries.linear_backward, p, index), {dx, dw, dbias});
}

// x, weight, residual, eps, out, sum, q8, scale
PyObject *rmsnorm(PyObject *const *a) {
  const Tensor &x = tensor(a[0], "x");
  const Tensor *weight = optional_tensor(a[1], "weight"), *residual = optional_tensor(a[2], "residual");
  const Tensor *out = optional_tensor(a[4], "out"), *sum = optional_tensor(a[5], "sum");
  const Tensor *scale = optional_tensor(a[7], "scale");
  if (sum && !residual) raise(PyExc_ValueError, "sum needs a residual: without one, h is x itself");
  need_2d(x, "x");
  const c10::DeviceIndex index = x.get_device();
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  const ScalarType type = x.scalar_type();
  phobos_rmsnorm_args_t p = {};
  p.type = need_float_type(type, "x");
  p.rows = x.size(0);
  p.cols = x.size(1);
  p.eps = static_cast<float>(PyFloat_AsDouble(a[3]));
  if (PyErr_Occurred()) throw Raised();
  const bool q8 = truth(a[6]);
  const ScalarType out_type = q8 ? ScalarType::Float8_e4m3fn : type;
  p.out_type = q8 ? PHOBOS_TYPE_E4M3 : p.type;
  p.x_row = row_stride(x, "x", p.rows, p.cols, type, index);
  p.x = x.data_ptr();
  if (weight) p.weight = vector(*weight, "weight", p.cols, type, index);
  if (residual) {
    p.residual_row = row_stride(*residual, "residual", p.rows, p.cols, type, index);
    p.residual = residual->data_ptr();
    if (sum) p.sum_row = row_stride(*sum, "sum", p.rows, p.cols, type, index);
  }
  if (out) p.out_row = row_stride(*out, "out", p.rows, p.cols, out_type, index);
  if (q8 && scale) vector(*scale, "scale", p.rows, ScalarType::Float, index);
  if (!q8) scale = nullptr;
  Tensor new_out, new_sum, new_scale;
  if (!out) {
    new_out = new_matrix(p.rows, p.cols, out_type, x);
    p.out_row = std::max<int64_t>(p.cols, 1);
    out = &new_out;
  }
  if (residual && !sum) {
    new_sum = new_matrix(p.rows, p.cols, type, x);
    p.sum_row = std::max<int64_t>(p.cols, 1);
    sum = &new_sum;
  }
  if (q8 && !scale) {
    new_scale = at::empty({p.rows}, at::TensorOptions().dtype(ScalarType::Float).device(x.device()));
    scale = &new_scale;
  }
  p.out = out->data_ptr();
  if (sum) p.sum = sum->data_ptr();
  if (scale) p.scale = static_cast<float *>(scale->data_ptr());
  for (const Tensor *t : {out, scale, sum}) written(t);
  return results(status(entries.rmsnorm, p, index), {out, scale, sum});
}

// dy, h, weight, dsum, eps, dx, dweight, need_dweight
PyObject *rmsnorm_backward(PyObject *const *a) {
  const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h");
  const Tensor *weight = optional_tensor(a[2], "weight"), *dsum = optional_tensor(a[3], "dsum");
  const Tensor *dx = optional_tensor(a[5], "dx"), *dweight = optional_tensor(a[6], "dweight");
  need_2d(h, "h");
  const c10::DeviceIndex index = h.get_device();
  const c10::cuda::OptionalCUDAGuard guard(h.device());
  const ScalarType type = h.scalar_type();
  phobos_rmsnorm_backward_args_t p = {};
  p.type = need_float_type(type, "h");
  p.rows = h.size(0);
  p.cols = h.size(1);
  p.eps = static_cast<float>(PyFloat_AsDouble(a[4]));
  if (PyErr_Occurred()) throw Raised();
  p.h_row = row_stride(h, "h", p.rows, p.cols, type, index);
  p.h = h.data_ptr();
  p.dy_row = row_stride(dy, "dy", p.rows, p.cols, type, index);
  p.dy = dy.data_ptr();
  if (weight) p.weight = vector(*weight, "weight", p.cols, type, index);
  if (dsum) {
    p.dsum_row = row_stride(*dsum, "dsum", p.rows, p.cols, type, index);
    p.dsum = dsum->data_ptr();
  }
  if (dx) p.dx_row = row_stride(*dx, "dx", p.rows, p.cols, type, index);
  const bool need_dweight = truth(a[7]);
  if (!need_dweight) dweight = nullptr;
  if (dweight) vector(*dweight, "dweight", p.cols, type, index);
  Tensor new_dx, new_dweight;
  if (!dx) {
    new_dx = new_matrix(p.rows, p.cols, type, h);
    p.dx_row = std::max<int64_t>(p.cols, 1);
    dx = &new_dx;
  }
  if (need_dweight && !dweight) {
    new_dweight = at::empty({p.cols}, at::TensorOptions().dtype(type).device(h.device()));
    dweight = &new_dweight;
  }
  p.dx = dx->data_ptr();
  if (dweight) p.dweight = dweight->data_ptr();
  for (const Tensor *t : {dx, dweight}) written(t);
  return results(status(entries.rmsnorm_backward, p, index), {dx, dweight});
}

PyObject *bind(PyObject *const *a) {
  entries.linear = reinterpret_cast<decltype(entries.linear)>(integer(a[0]));
  entries.linear_backward = reinterpret_cast<decltype(entries.linear_backward)>(integer(a[1]));
  entries.rmsnorm = reinterpret_cast<decltype(entries.rmsnorm)>(integer(a[2]));
  entries.rmsnorm_backward = reinterpret_cast<decltype(entries.rmsnorm_backward)>(integer(a[3]));
  Py_RETURN_NONE;
}

// C++ exceptions (torch's among them) become Python ones.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *function(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return F(args);
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&function<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<linear, 12>("linear"),
                         method<linear_backward, 14>("linear_backward"),
                         method<rmsnorm, 8>("rmsnorm"),
                         method<rmsnorm_backward, 8>("rmsnorm_backward"),
                         method<bind, 4>("bind"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_binding() { return PyModule_Create(&module); }
