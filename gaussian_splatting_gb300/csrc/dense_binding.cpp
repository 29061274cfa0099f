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
#include <vector>

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
  return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat8_e4m3fn ? "torch.float8_e4m3fn" : at::toString(t);
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

// Bits of the indices of `rows` rows (any number of them if negative).
int index_bits(const at::Tensor& t, int64_t rows, const at::Tensor& like) {
  const at::ScalarType s = t.scalar_type();
  if ((s != at::kInt && s != at::kLong) || t.device() != like.device() || t.dim() != 1 || (rows >= 0 && t.size(0) != rows) ||
      (t.size(0) > 1 && t.stride(0) != 1))
    throw Refused{"idx must be a contiguous int32 or int64 vector" + (rows >= 0 ? " of " + std::to_string(rows) : std::string()) +
                  " on " + like.device().str() + ", got " + type_name(s) + " " + text(t) + " on " + t.device().str()};
  return s == at::kInt ? 32 : 64;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) throw python_error();
  return v;
}

// (table, idx, scale, out, stream) -> y
PyObject* embedding_fwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(5)
  const at::Tensor &table = tensor(o[0], "table"), &idx = tensor(o[1], "idx");
  gs_embedding_desc d{};
  d.dtype = dtype_of(table, "table");
  d.index_bits = index_bits(idx, -1, table);
  const int64_t n = table.size(0), width = table.size(1), rows = idx.size(0);
  if (width > INT32_MAX) throw Refused{"too many features"};
  d.rows = rows, d.n = n, d.width = (int32_t)width, d.scale = (float)number(o[2]);
  d.ldt = matrix(table, "table", n, width, table);
  Maybe y = maybe(o[3], "out");
  On on(table, o[4]);
  if (!y) y = empty({rows, width}, table.scalar_type(), table);
  d.ldy = matrix(*y, "out", rows, width, table);
  call("gs_embedding_fwd", [&] { return gs_embedding_fwd(&d, table.data_ptr(), idx.data_ptr(), y->data_ptr(), on.stream); });
  return THPVariable_Wrap(*y);
  GS_END
}

// (dy, idx, n, scale, dtable, stream) -> dtable
PyObject* embedding_bwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(6)
  const at::Tensor &dy = tensor(o[0], "dy"), &idx = tensor(o[1], "idx");
  gs_embedding_desc d{};
  d.dtype = dtype_of(dy, "dy");
  const int64_t rows = dy.size(0), width = dy.size(1), n = integer(o[2]);
  d.index_bits = index_bits(idx, rows, dy);
  if (width > INT32_MAX) throw Refused{"too many features"};
  if (n < 0) throw Refused{"n must be >= 0, got " + std::to_string(n)};
  d.rows = rows, d.n = n, d.width = (int32_t)width, d.scale = (float)number(o[3]);
  d.ldy = matrix(dy, "dy", rows, width, dy);
  Maybe dtable = maybe(o[4], "dtable");
  On on(dy, o[5]);
  if (!dtable) dtable = empty({n, width}, dy.scalar_type(), dy);
  d.ldt = matrix(*dtable, "dtable", n, width, dy);
  const size_t need = gs_embedding_bwd_workspace_size(&d);
  Maybe ws;
  if (need) ws = empty({(int64_t)need}, at::kByte, dy);
  call("gs_embedding_bwd", [&] {
    return gs_embedding_bwd(&d, dy.data_ptr(), idx.data_ptr(), dtable->data_ptr(), at(ws), need, on.stream);
  });
  return THPVariable_Wrap(*dtable);
  GS_END
}

// samples maps of equally many rows
void maps(gs_groupnorm_desc& d, int64_t rows, int64_t width, int64_t samples, int64_t groups) {
  if (width > INT32_MAX) throw Refused{"too many features"};
  if (samples < 0 || samples > INT32_MAX || (samples == 0 ? rows != 0 : rows % samples != 0))
    throw Refused{std::to_string(rows) + " rows are not " + std::to_string(samples) + " maps of equal size"};
  if (groups < 1 || groups > width || width % groups != 0)
    throw Refused{std::to_string(width) + " channels do not form " + std::to_string(groups) + " groups"};
  d.samples = samples, d.rows = samples ? rows / samples : 0, d.width = (int32_t)width, d.groups = (int32_t)groups;
}

// (x, gamma, beta, groups, samples, act, eps, out, stats, stream) -> (y, mean, rstd)
PyObject* groupnorm_fwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(10)
  const at::Tensor &x = tensor(o[0], "x"), &gamma = tensor(o[1], "gamma"), &beta = tensor(o[2], "beta");
  gs_groupnorm_desc d{};
  d.dtype = dtype_of(x, "x");
  const int64_t rows = x.size(0), n = x.size(1);
  maps(d, rows, n, integer(o[4]), integer(o[3]));
  d.act = (int32_t)integer(o[5]), d.eps = (float)number(o[6]);
  d.ldx = matrix(x, "x", rows, n, x);
  vector(gamma, "gamma", n, x);
  vector(beta, "beta", n, x);
  On on(x, o[9]);
  Maybe y = maybe(o[7], "out"), mean, rstd;
  if (!y) y = empty({rows, n}, x.scalar_type(), x);
  d.ldy = matrix(*y, "out", rows, n, x);
  if (PyObject_IsTrue(o[8]) > 0)
    mean = empty({d.samples, d.groups}, at::kFloat, x), rstd = empty({d.samples, d.groups}, at::kFloat, x);
  const size_t need = gs_groupnorm_fwd_workspace_size(&d);
  Maybe ws;
  if (need) ws = empty({(int64_t)need}, at::kByte, x);
  call("gs_groupnorm_fwd", [&] {
    return gs_groupnorm_fwd(&d, x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), y->data_ptr(), static_cast<float*>(at(mean)),
                            static_cast<float*>(at(rstd)), at(ws), need, on.stream);
  });
  return wrap_all(y, mean, rstd, 3);
  GS_END
}

// (dy, x, gamma, beta, mean, rstd, act, skip, dx, dgamma, dbeta, need_dx, need_dparams, stream) -> (dx, dgamma, dbeta)
PyObject* groupnorm_bwd(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(14)
  const at::Tensor &dy = tensor(o[0], "dy"), &x = tensor(o[1], "x"), &gamma = tensor(o[2], "gamma"), &beta = tensor(o[3], "beta");
  const at::Tensor &mean = tensor(o[4], "mean"), &rstd = tensor(o[5], "rstd");
  const Maybe skip = maybe(o[7], "skip");
  gs_groupnorm_desc d{};
  d.dtype = dtype_of(dy, "dy");
  const int64_t rows = dy.size(0), n = dy.size(1);
  for (const auto& [t, name] : {std::pair<const at::Tensor&, const char*>(mean, "mean"), {rstd, "rstd"}})
    if (t.scalar_type() != at::kFloat || t.device() != dy.device() || t.dim() != 2 || t.sizes() != mean.sizes() || !t.is_contiguous())
      throw Refused{std::string(name) + " must be a contiguous float32 matrix [samples, groups] on " + dy.device().str() + ", got " +
                    text(t)};
  maps(d, rows, n, mean.size(0), mean.size(1));
  d.act = (int32_t)integer(o[6]);
  d.lddy = matrix(dy, "dy", rows, n, dy), d.ldx = matrix(x, "x", rows, n, dy);
  vector(gamma, "gamma", n, dy);
  vector(beta, "beta", n, dy);
  if (skip) d.ldskip = matrix(*skip, "skip", rows, n, dy);
  On on(dy, o[13]);
  Maybe dx = maybe(o[8], "dx"), dgamma = maybe(o[9], "dgamma"), dbeta = maybe(o[10], "dbeta");
  if (!dx && PyObject_IsTrue(o[11]) > 0) dx = empty({rows, n}, dy.scalar_type(), dy);
  if (!dgamma && PyObject_IsTrue(o[12]) > 0) dgamma = empty({n}, dy.scalar_type(), dy);
  if (!dbeta && PyObject_IsTrue(o[12]) > 0) dbeta = empty({n}, dy.scalar_type(), dy);
  if (dx) d.lddx = matrix(*dx, "dx", rows, n, dy);
  if (dgamma) vector(*dgamma, "dgamma", n, dy);
  if (dbeta) vector(*dbeta, "dbeta", n, dy);
  const size_t need = dx || dgamma || dbeta ? gs_groupnorm_bwd_workspace_size(&d) : 0;
  Maybe ws;
  if (need) ws = empty({(int64_t)need}, at::kByte, dy);
  call("gs_groupnorm_bwd", [&] {
    return gs_groupnorm_bwd(&d, dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), beta.data_ptr(),
                            static_cast<const float*>(mean.data_ptr()), static_cast<const float*>(rstd.data_ptr()), at(skip), at(dx),
                            at(dgamma), at(dbeta), at(ws), need, on.stream);
  });
  return wrap_all(dx, dgamma, dbeta, 3);
  GS_END
}

// A list or tuple (or anything that iterates) of `count` entries; no entries at all where it is None.
struct Sequence {
  PyObject* fast = nullptr;
  Py_ssize_t n = 0;
  Sequence(PyObject* o, const char* name, Py_ssize_t count) {
    if (o == Py_None) return;
    fast = PySequence_Fast(o, "not a sequence");
    if (!fast) {
      PyErr_Clear();
      throw Refused{std::string(name) + " must be a sequence of tensors"};
    }
    n = PySequence_Fast_GET_SIZE(fast);
    if (count >= 0 && n != count) {
      const std::string what = std::string(name) + " must have " + std::to_string(count) + " entries, got " + std::to_string(n);
      Py_DECREF(fast);
      throw Refused{what};
    }
  }
  Sequence(const Sequence&) = delete;
  ~Sequence() { Py_XDECREF(fast); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// one tensor of an update
const at::Tensor& member(const Sequence& s, Py_ssize_t i, const char* name, const at::Tensor* like, at::ScalarType type) {
  const at::Tensor& t = tensor(s[i], name);
  if (t.scalar_type() != type || (like && (t.device() != like->device() || t.sizes() != like->sizes())) || !t.is_contiguous())
    throw Refused{std::string(name) + "[" + std::to_string(i) + "] must be a contiguous " + type_name(type) + " tensor" +
                  (like ? " " + text(*like) + " on " + like->device().str() : std::string()) + ", got " + type_name(t.scalar_type()) +
                  " " + text(t) + " on " + t.device().str()};
  return t;
}
// a number for all of them, or a sequence of one for each
std::vector<double> numbers(PyObject* o, const char* name, Py_ssize_t count) {
  if (PyFloat_Check(o) || PyLong_Check(o)) return std::vector<double>(count, number(o));
  const Sequence s(o, name, count);
  if (!s.fast) throw Refused{std::string(name) + " must be a number or a sequence of them"};
  std::vector<double> v(count);
  for (Py_ssize_t i = 0; i < count; ++i) v[i] = number(s[i]);
  return v;
}

// (params, grads, exp_avg, exp_avg_sq, step, lr, beta1, beta2, eps, weight_decay, scales or None, copies, seed, counts, stream)
PyObject* adamw(PyObject*, PyObject* const* o, Py_ssize_t count) {
  GS_BEGIN(15)
  const Sequence params(o[0], "params", -1);
  const Py_ssize_t n = params.n;
  if (n > INT32_MAX) throw Refused{"too many tensors"};
  const Sequence grads(o[1], "grads", n), m(o[2], "exp_avg", n), v(o[3], "exp_avg_sq", n), copies(o[11], "copies", n);
  const Sequence scales(o[10], "scales", 2);
  const Sequence ms(scales.fast ? scales[0] : Py_None, "scales[0]", n), vs(scales.fast ? scales[1] : Py_None, "scales[1]", n);
  if (n && (!grads.fast || !m.fast || !v.fast)) throw Refused{"grads, exp_avg and exp_avg_sq must be sequences of tensors"};
  if (n && scales.fast && (!ms.fast || !vs.fast)) throw Refused{"scales must be two sequences of tensors"};
  gs_adamw_desc d{};
  d.step = integer(o[4]), d.beta1 = number(o[6]), d.beta2 = number(o[7]), d.eps = number(o[8]);
  d.state_bits = scales.fast ? 8 : 32;
  d.seed = (uint32_t)PyLong_AsUnsignedLongLongMask(o[12]);
  if (PyErr_Occurred()) throw python_error();
  const std::vector<double> lr = numbers(o[5], "lr", n), decay = numbers(o[9], "weight_decay", n);
  std::vector<gs_adamw_tensor> all(n);
  const at::Tensor* first = nullptr;
  at::ScalarType grad_type = at::kFloat;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor& p = member(params, i, "params", nullptr, at::kFloat);
    if (!p.is_cuda()) throw Refused{"params must be CUDA tensors: there is no CPU path"};
    if (!first) {
      first = &p;
      grad_type = tensor(grads[0], "grads").scalar_type();
      if (grad_type != at::kFloat && grad_type != at::kBFloat16)
        throw Refused{std::string("grads must be float32 or bfloat16, got ") + type_name(grad_type)};
    } else if (p.device() != first->device()) {
      throw Refused{"params must be on one device, got " + first->device().str() + " and " + p.device().str()};
    }
    const at::ScalarType state = scales.fast ? at::kFloat8_e4m3fn : at::kFloat;
    gs_adamw_tensor& t = all[i];
    t.param = static_cast<float*>(p.data_ptr());
    t.grad = member(grads, i, "grads", &p, grad_type).data_ptr();
    t.exp_avg = member(m, i, "exp_avg", &p, state).data_ptr();
    t.exp_avg_sq = member(v, i, "exp_avg_sq", &p, state).data_ptr();
    if (scales.fast) {
      for (const auto& [s, name] : {std::pair<const Sequence&, const char*>(ms, "scales[0]"), {vs, "scales[1]"}}) {
        const at::Tensor& c = tensor(s[i], name);
        if (c.scalar_type() != at::kFloat || c.device() != p.device() || c.dim() != 1 || c.size(0) != (p.numel() + 255) / 256 ||
            !c.is_contiguous())
          throw Refused{std::string(name) + "[" + std::to_string(i) + "] must be a contiguous float32 vector of " +
                        std::to_string((p.numel() + 255) / 256) + " on " + p.device().str() + ", got " + text(c)};
        (&s == &ms ? t.exp_avg_scale : t.exp_avg_sq_scale) = static_cast<float*>(c.data_ptr());
      }
    }
    if (copies.fast) t.copy = member(copies, i, "copies", &p, at::kBFloat16).data_ptr();
    t.n = p.numel(), t.lr = lr[i], t.weight_decay = decay[i];
  }
  d.grad_dtype = grad_type == at::kFloat ? GS_F32 : GS_BF16;
  if (!first) Py_RETURN_NONE;
  const int64_t* counts = nullptr;
  int n_counts = 0;
  if (o[13] != Py_None) {
    const at::Tensor& c = tensor(o[13], "counts");
    if (c.scalar_type() != at::kLong || c.device() != first->device() || c.dim() != 2 || c.size(1) != 2 || !c.is_contiguous() ||
        c.size(0) > INT32_MAX)
      throw Refused{"counts must be a contiguous int64 matrix [records, 2] on " + first->device().str() + ", got " + text(c)};
    counts = static_cast<const int64_t*>(c.data_ptr()), n_counts = (int)c.size(0);
  }
  On on(*first, o[14]);
  call("gs_adamw", [&] { return gs_adamw(&d, all.data(), (int)n, counts, n_counts, on.stream); });
  Py_RETURN_NONE;
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
                         GS_METHOD(embedding_fwd), GS_METHOD(embedding_bwd), GS_METHOD(groupnorm_fwd), GS_METHOD(groupnorm_bwd),
                         GS_METHOD(adamw),        GS_METHOD(check_matrix), GS_METHOD(check_vector), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__dense() { return PyModule_Create(&module); }
