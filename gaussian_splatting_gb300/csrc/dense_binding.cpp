// Python functions over the dense-layer entry points for torch tensors (module _dense, used by dense.py): argument
// checks, allocation of the outputs that the caller did not hand in and of the workspace, the stream, the call.
//
// A small layer's kernels take 4 to 10 us.  A call takes 3.4 us of host time here for the linear forward, 6.9 for its
// backward and 5.0 for the norm; through torch.empty and ctypes, without any checks, 12.7, 19.9 and 20.6.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/gs.h"

namespace {

// An argument that a call cannot take: becomes a ValueError.
struct Refused {
  std::string what;
};
// A call that returned an error: becomes a GSError.
struct Failed {
  int status;
  const char* where;
};

std::string text(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

const char* type_name(at::ScalarType t) {
  return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : at::toString(t);
}

void check_like(const at::Tensor& t, const char* name, const at::Tensor& like) {
  if (t.scalar_type() != like.scalar_type() || t.device() != like.device())
    throw Refused{std::string(name) + " must be " + type_name(like.scalar_type()) + " on " + like.device().str() + ", got " +
                  type_name(t.scalar_type()) + " on " + t.device().str()};
}

// Row stride of a matrix argument, checked against the call's shape, type and device.
int64_t matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t cols, const at::Tensor& like) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    throw Refused{std::string(name) + " must have shape [" + std::to_string(rows) + ", " + std::to_string(cols) + "], got " +
                  text(t)};
  check_like(t, name, like);
  if (cols > 1 && t.stride(1) != 1) throw Refused{std::string(name) + " must have unit stride along its rows"};
  if (rows <= 1) return cols;
  if (t.stride(0) < cols)
    throw Refused{std::string(name) + " has overlapping rows (stride " + std::to_string(t.stride(0)) + " < " +
                  std::to_string(cols) + ")"};
  return t.stride(0);
}

void vector(const at::Tensor& t, const char* name, int64_t n, const at::Tensor& like) {
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    throw Refused{std::string(name) + " must be a contiguous vector of " + std::to_string(n) + ", got " + text(t)};
  check_like(t, name, like);
}

void statistic(const at::Tensor& t, const char* name, int64_t rows, const at::Tensor& like) {
  if (t.scalar_type() != at::kFloat || t.device() != like.device() || t.dim() != 1 || t.size(0) != rows ||
      (rows > 1 && t.stride(0) != 1))
    throw Refused{std::string(name) + " must be a contiguous float32 vector of " + std::to_string(rows) + " on " +
                  like.device().str()};
}

// The element type of the argument that sets the call's shape.
int dtype_of(const at::Tensor& t, const char* name) {
  const at::ScalarType s = t.scalar_type();
  if (s != at::kFloat && s != at::kBFloat16)
    throw Refused{std::string(name) + " must be float32 or bfloat16, got " + type_name(s)};
  if (t.dim() != 2) throw Refused{std::string(name) + " must be a matrix, got " + text(t)};
  if (!t.is_cuda()) throw Refused{std::string(name) + " must be a CUDA tensor: there is no CPU path"};
  return s == at::kFloat ? GS_F32 : GS_BF16;
}

using Maybe = std::optional<at::Tensor>;

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
Maybe maybe(PyObject* o, const char* name) { return o == Py_None ? Maybe() : Maybe(tensor(o, name)); }
void* at(const Maybe& t) { return t ? t->data_ptr() : nullptr; }

int32_t* status_at(PyObject* o, const at::Tensor& like) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "status");
  if (t.scalar_type() != at::kInt || t.device() != like.device() || t.numel() < 1)
    throw Refused{"status must be an int32 tensor on " + like.device().str()};
  return static_cast<int32_t*>(t.data_ptr());
}

// The tensors' device and the call's stream (None: the current one) as torch's current ones.
struct On {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  cudaStream_t stream;
  On(const at::Tensor& like, PyObject* handle) : device(like.device()) {
    if (handle == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(like.device().index()).stream();
    } else {
      stream = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(handle));
      if (PyErr_Occurred()) throw python_error();
      guard.emplace(c10::cuda::getStreamFromExternal(stream, like.device().index()));
    }
  }
};

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}

template <typename F>
void call(const char* where, F f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  if (status) throw Failed{status, where};
}

PyObject* wrap(Maybe& t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}
PyObject* wrap_all(Maybe a, Maybe b, Maybe c, int n) {
  PyObject* tuple = PyTuple_New(n);
  if (!tuple) return nullptr;
  Maybe* all[3] = {&a, &b, &c};
  for (int i = 0; i < n; ++i) {
    PyObject* o = wrap(*all[i]);
    if (!o) {
      Py_DECREF(tuple);
      return nullptr;
    }
    PyTuple_SET_ITEM(tuple, i, o);
  }
  return tuple;
}

void raise_failed(const Failed& f) {
  PyObject* native = PyImport_ImportModule("gaussian_splatting_gb300._native");
  PyObject* type = native ? PyObject_GetAttrString(native, "GSError") : nullptr;
  PyObject* error = type ? PyObject_CallFunction(type, "iss", f.status, f.where, gs_last_error()) : nullptr;
  if (error) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(native);
}

#define GS_BEGIN(N)                                                                     \
  HANDLE_TH_ERRORS                                                                      \
  try {                                                                                 \
    if (count != N) throw Refused{"expected " #N " arguments, got " + std::to_string(count)};
#define GS_END                                        \
  } catch (const Refused& r) {                        \
    PyErr_SetString(PyExc_ValueError, r.what.c_str()); \
    return nullptr;                                   \
  } catch (const Failed& f) {                         \
    raise_failed(f);                                  \
    return nullptr;                                   \
  }                                                   \
  END_HANDLE_TH_ERRORS

// (x, w, bias, residual, act, keep_z, out, z, status, stream) -> (y, z)
PyObject* linear_fwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(10)
  const at::Tensor &x = tensor(o[0], "x"), &w = tensor(o[1], "w");
  const Maybe bias = maybe(o[2], "bias"), residual = maybe(o[3], "residual");
  gs_linear_desc d{};
  d.dtype = dtype_of(x, "x");
  if (w.dim() != 2) throw Refused{"w must be a matrix, got " + text(w)};
  const int64_t rows = x.size(0), in = x.size(1), out = w.size(0);
  if (in > INT32_MAX || out > INT32_MAX) throw Refused{"too many features"};
  d.rows = rows, d.in_features = (int32_t)in, d.out_features = (int32_t)out, d.act = (int32_t)PyLong_AsLong(o[4]);
  d.ldx = matrix(x, "x", rows, in, x), d.ldw = matrix(w, "w", out, in, x);
  if (bias) vector(*bias, "bias", out, x);
  if (residual) d.ldr = matrix(*residual, "residual", rows, out, x);
  int32_t* status = status_at(o[8], x);
  On on(x, o[9]);
  Maybe y = maybe(o[6], "out"), z = maybe(o[7], "z");
  if (!y) y = empty({rows, out}, x.scalar_type(), x);
  d.ldy = matrix(*y, "out", rows, out, x);
  if (!z && PyObject_IsTrue(o[5]) > 0) z = empty({rows, out}, x.scalar_type(), x);
  if (z) d.ldz = matrix(*z, "z", rows, out, x);
  const size_t need = gs_linear_fwd_workspace_size(&d);
  Maybe ws;
  if (need) ws = empty({(int64_t)need}, at::kByte, x);
  call("gs_linear_fwd", [&] {
    return gs_linear_fwd(&d, x.data_ptr(), w.data_ptr(), at(bias), at(residual), y->data_ptr(), at(z), at(ws), need, status,
                         on.stream);
  });
  return wrap_all(y, z, Maybe(), 2);
  GS_END
}

// (dy, x, w, z, act, bias, dx, dw, dbias, need_dx, need_dw, status, stream) -> (dx, dw, dbias)
PyObject* linear_bwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(13)
  const at::Tensor &dy = tensor(o[0], "dy"), &x = tensor(o[1], "x"), &w = tensor(o[2], "w");
  Maybe z = maybe(o[3], "z");
  gs_linear_desc d{};
  d.dtype = dtype_of(dy, "dy");
  if (x.dim() != 2) throw Refused{"x must be a matrix, got " + text(x)};
  const int64_t rows = dy.size(0), out = dy.size(1), in = x.size(1);
  if (in > INT32_MAX || out > INT32_MAX) throw Refused{"too many features"};
  d.rows = rows, d.in_features = (int32_t)in, d.out_features = (int32_t)out, d.act = (int32_t)PyLong_AsLong(o[4]);
  d.ldy = matrix(dy, "dy", rows, out, dy), d.ldx = matrix(x, "x", rows, in, dy), d.ldw = matrix(w, "w", out, in, dy);
  if (d.act == GS_ACT_NONE) z.reset();
  else if (!z) throw Refused{"z is needed for the gradient of an activation"};
  else d.ldz = matrix(*z, "z", rows, out, dy);
  int32_t* status = status_at(o[11], dy);
  On on(dy, o[12]);
  Maybe dx = maybe(o[6], "dx"), dw = maybe(o[7], "dw"), db = maybe(o[8], "dbias");
  if (!dx && PyObject_IsTrue(o[9]) > 0) dx = empty({rows, in}, dy.scalar_type(), dy);
  if (!dw && PyObject_IsTrue(o[10]) > 0) dw = empty({out, in}, dy.scalar_type(), dy);
  if (!db && PyObject_IsTrue(o[5]) > 0) db = empty({out}, dy.scalar_type(), dy);
  if (dx) d.lddx = matrix(*dx, "dx", rows, in, dy);
  if (dw) d.lddw = matrix(*dw, "dw", out, in, dy);
  if (db) vector(*db, "dbias", out, dy);
  const size_t need = gs_linear_bwd_workspace_size(&d);
  Maybe ws;
  if (need) ws = empty({(int64_t)need}, at::kByte, dy);
  call("gs_linear_bwd", [&] {
    return gs_linear_bwd(&d, dy.data_ptr(), x.data_ptr(), w.data_ptr(), at(z), at(dx), at(dw), at(db), at(ws), need, status,
                         on.stream);
  });
  return wrap_all(dx, dw, db, 3);
  GS_END
}

// (x, gamma, beta, eps, out, stats, stream) -> (y, mean, rstd)
PyObject* layernorm_fwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(7)
  const at::Tensor &x = tensor(o[0], "x"), &gamma = tensor(o[1], "gamma"), &beta = tensor(o[2], "beta");
  gs_layernorm_desc d{};
  d.dtype = dtype_of(x, "x");
  const int64_t rows = x.size(0), n = x.size(1);
  if (n > INT32_MAX) throw Refused{"too many features"};
  d.rows = rows, d.width = (int32_t)n, d.eps = (float)PyFloat_AsDouble(o[3]);
  if (PyErr_Occurred()) return nullptr;
  d.ldx = matrix(x, "x", rows, n, x);
  vector(gamma, "gamma", n, x);
  vector(beta, "beta", n, x);
  On on(x, o[6]);
  Maybe y = maybe(o[4], "out"), mean, rstd;
  if (!y) y = empty({rows, n}, x.scalar_type(), x);
  d.ldy = matrix(*y, "out", rows, n, x);
  if (PyObject_IsTrue(o[5]) > 0) mean = empty({rows}, at::kFloat, x), rstd = empty({rows}, at::kFloat, x);
  call("gs_layernorm_fwd", [&] {
    return gs_layernorm_fwd(&d, x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), y->data_ptr(), static_cast<float*>(at(mean)),
                            static_cast<float*>(at(rstd)), on.stream);
  });
  return wrap_all(y, mean, rstd, 3);
  GS_END
}

// (dy, x, gamma, mean, rstd, skip, dx, dgamma, dbeta, need_dx, need_dparams, stream) -> (dx, dgamma, dbeta)
PyObject* layernorm_bwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(12)
  const at::Tensor &dy = tensor(o[0], "dy"), &x = tensor(o[1], "x"), &gamma = tensor(o[2], "gamma");
  const at::Tensor &mean = tensor(o[3], "mean"), &rstd = tensor(o[4], "rstd");
  const Maybe skip = maybe(o[5], "skip");
  gs_layernorm_desc d{};
  d.dtype = dtype_of(dy, "dy");
  const int64_t rows = dy.size(0), n = dy.size(1);
  if (n > INT32_MAX) throw Refused{"too many features"};
  d.rows = rows, d.width = (int32_t)n;
  d.lddy = matrix(dy, "dy", rows, n, dy), d.ldx = matrix(x, "x", rows, n, dy);
  vector(gamma, "gamma", n, dy);
  statistic(mean, "mean", rows, dy);
  statistic(rstd, "rstd", rows, dy);
  if (skip) d.ldskip = matrix(*skip, "skip", rows, n, dy);
  On on(dy, o[11]);
  Maybe dx = maybe(o[6], "dx"), dgamma = maybe(o[7], "dgamma"), dbeta = maybe(o[8], "dbeta");
  if (!dx && PyObject_IsTrue(o[9]) > 0) dx = empty({rows, n}, dy.scalar_type(), dy);
  if (!dgamma && PyObject_IsTrue(o[10]) > 0) dgamma = empty({n}, dy.scalar_type(), dy);
  if (!dbeta && PyObject_IsTrue(o[10]) > 0) dbeta = empty({n}, dy.scalar_type(), dy);
  if (dx) d.lddx = matrix(*dx, "dx", rows, n, dy);
  if (dgamma) vector(*dgamma, "dgamma", n, dy);
  if (dbeta) vector(*dbeta, "dbeta", n, dy);
  const size_t need = dgamma || dbeta ? gs_layernorm_bwd_workspace_size(&d) : 0;
  Maybe ws;
  if (need) ws = empty({(int64_t)need}, at::kByte, dy);
  call("gs_layernorm_bwd", [&] {
    return gs_layernorm_bwd(&d, dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), static_cast<const float*>(mean.data_ptr()),
                            static_cast<const float*>(rstd.data_ptr()), at(skip), at(dx), at(dgamma), at(dbeta), at(ws), need,
                            on.stream);
  });
  return wrap_all(dx, dgamma, dbeta, 3);
  GS_END
}

// The argument checks by themselves: (tensor, name, rows, cols, like) -> row stride; (tensor, name, n, like) -> None
PyObject* check_matrix(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(5)
  return PyLong_FromLongLong(matrix(tensor(o[0], "tensor"), PyUnicode_AsUTF8(o[1]), PyLong_AsLongLong(o[2]),
                                    PyLong_AsLongLong(o[3]), tensor(o[4], "like")));
  GS_END
}
PyObject* check_vector(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(4)
  vector(tensor(o[0], "tensor"), PyUnicode_AsUTF8(o[1]), PyLong_AsLongLong(o[2]), tensor(o[3], "like"));
  Py_RETURN_NONE;
  GS_END
}

#define GS_METHOD(F) {#F, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GS_METHOD(linear_fwd),   GS_METHOD(linear_bwd),   GS_METHOD(layernorm_fwd), GS_METHOD(layernorm_bwd),
                         GS_METHOD(check_matrix), GS_METHOD(check_vector), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__dense() { return PyModule_Create(&module); }
