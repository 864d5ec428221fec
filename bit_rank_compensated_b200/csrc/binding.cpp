// The Python calls of the operators around the projections: checks of their tensors, outputs and scratch
// from torch's allocator, and the call of the C ABI on the tensors' device and its current stream.
//
// A small call's time is its caller's: the same steps in Python with ctypes took 11 to 24 us of the host
// for kernels of 2 to 10 us. The entry points' addresses come from the loaded libsvdq.so
// (bind), so this module links to torch alone. A call returns its outputs, or the svdq_status (an int)
// that the library refused it with; what it refuses itself is a ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "svdq.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string &what) { throw Refused(what); }

struct Entry {
  decltype(&svdq_layer_norm) layer_norm = nullptr;
  decltype(&svdq_layer_norm_workspace_bytes) layer_norm_workspace_bytes = nullptr;
  decltype(&svdq_layer_norm_backward) layer_norm_backward = nullptr;
  decltype(&svdq_i8_quantize_rows) i8_quantize_rows = nullptr;
  decltype(&svdq_i8_layer_norm_quantize) i8_layer_norm_quantize = nullptr;
  decltype(&svdq_i8_workspace_bytes) i8_workspace_bytes = nullptr;
  decltype(&svdq_i8_gemm) i8_gemm = nullptr;
  decltype(&svdq_i8_linear_forward) i8_linear_forward = nullptr;
  decltype(&svdq_rope_axes_table) rope_axes_table = nullptr;
  decltype(&svdq_rope_axes_apply) rope_axes_apply = nullptr;
} entry;

// ---------------------------------------------------------------- arguments
bool has(PyObject *o) { return o != Py_None; }

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  const Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  // (of a conjugated tensor's imaginary part: its memory holds the other sign)
  if (t.is_neg()) refuse(std::string(name) + " must not be a lazily negated view (resolve_neg() makes a plain tensor of it)");
  return t;
}

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return SVDQ_BF16;
    case at::kHalf: return SVDQ_F16;
    case at::kFloat: return SVDQ_F32;
    case at::kInt: return SVDQ_I32;
    case at::kLong: return SVDQ_I64;
    default: return -1;
  }
}
int float_code(const Tensor &t, const char *name) {
  const int c = dtype_code(t.scalar_type());
  if (c < 0 || c > SVDQ_F32) refuse(std::string(name) + " must be of bf16, fp16 or fp32");
  return c;
}

int count(int64_t n, const char *name) {
  if (n < 0 || n > INT32_MAX) refuse(std::string(name) + " is out of range");
  return static_cast<int>(n);
}

// A matrix with contiguous rows.
struct Rows {
  int M, K;
  size_t stride;
};
Rows rows_of(const Tensor &t, const char *name) {
  if (t.dim() != 2) refuse(std::string(name) + " must have two dimensions");
  const int64_t M = t.size(0), K = t.size(1);
  const int64_t stride = M > 1 ? t.stride(0) : K;
  if ((K > 1 && t.stride(1) != 1) || stride < K) refuse("the rows of " + std::string(name) + " must be contiguous and must not overlap");
  return {count(M, name), count(K, name), static_cast<size_t>(stride)};
}

// n contiguous values of a type on a device; their address.
void *values(PyObject *o, const char *name, int64_t n, at::ScalarType type, const at::Device &device) {
  const Tensor &t = tensor(o, name);
  if (t.scalar_type() != type || t.numel() != n || t.device() != device || !t.is_contiguous())
    refuse(std::string(name) + " must be " + std::to_string(n) + " contiguous values of " + c10::toString(type) + " on " + device.str());
  return t.data_ptr();
}
const float *floats(PyObject *o, const char *name, int64_t n, const at::Device &device) {
  return has(o) ? static_cast<const float *>(values(o, name, n, at::kFloat, device)) : nullptr;
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Device &device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

// A caller's M x K output of a type, or none; its rows' distance either way.
Tensor output(PyObject *o, const char *name, const Rows &r, const Tensor &like, size_t *stride) {
  if (!has(o)) {
    *stride = static_cast<size_t>(r.K);
    return {};
  }
  const Tensor &t = tensor(o, name);
  const Rows q = rows_of(t, name);
  if (q.M != r.M || q.K != r.K || t.scalar_type() != like.scalar_type() || t.device() != like.device())
    refuse(std::string(name) + " must have X's shape, type and device");
  *stride = q.stride;
  return t;
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v == 1;
}

// While a call allocates and launches, other threads may run Python: an allocation can be slow, and a launch can wait for a
// full queue, whose next entry may be a host function that needs the interpreter. Nothing in its scope touches a
// Python object.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

void *stream_of(const at::Device &d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

// Weight and bias ([K] or [groups, K]) of a layer norm.
svdq_norm_affine affine_of(const Tensor &X, const Rows &r, PyObject *weight, PyObject *bias, int64_t rows_per_group,
                           float offset, int64_t groups) {
  svdq_norm_affine a{};
  int64_t n = groups;
  a.dtype = SVDQ_F32;
  bool first = true;
  for (int i = 0; i < 2; ++i) {
    PyObject *o = i ? bias : weight;
    if (!has(o)) continue;
    const char *name = i ? "bias" : "weight";
    const Tensor &t = tensor(o, name);
    const int code = float_code(t, name);
    int64_t g = 1, stride = r.K, columns = 0;
    if (t.dim() == 1) {
      columns = t.size(0);
      if (columns > 1 && t.stride(0) != 1) refuse(std::string(name) + " must be contiguous");
    } else {
      const Rows q = rows_of(t, name);
      g = q.M, columns = q.K, stride = static_cast<int64_t>(q.stride);
    }
    if (columns != r.K || t.device() != X.device() || (n > 0 && g != n) || (!first && code != a.dtype))
      refuse("weight and bias must be of one type and shape, with X's columns, on X's device");
    first = false;
    n = g;
    a.dtype = code;
    (i ? a.bias : a.weight) = t.data_ptr();
    (i ? a.bias_stride : a.weight_stride) = static_cast<size_t>(stride);
    if (g < 1) refuse("no groups");
  }
  if (n < 1) n = 1;
  int64_t rows = rows_per_group;
  if (rows == 0) rows = (r.M + n - 1) / n;
  if (rows == 0) rows = 1;
  if (rows < 1 || rows > INT32_MAX || n > INT32_MAX || n * rows < r.M)
    refuse(std::to_string(n) + " groups of " + std::to_string(rows) + " rows do not cover " + std::to_string(r.M) + " rows");
  a.groups = static_cast<int32_t>(n);
  a.rows_per_group = static_cast<int32_t>(rows);
  a.weight_offset = offset;
  return a;
}

// A caller's workspace, or one of `need` bytes.
struct Space {
  Tensor kept;
  void *data = nullptr;
  size_t bytes = 0;

  void make(size_t need, const at::Device &device) {
    if (!kept.defined() && need > 0) kept = fresh({static_cast<int64_t>(need)}, at::kByte, device);
    if (kept.defined()) {
      data = kept.data_ptr();
      bytes = kept.nbytes();
    }
  }
};
Space space_of(PyObject *o, const at::Device &device) {
  Space s;
  if (has(o)) {
    s.kept = tensor(o, "workspace");
    if (s.kept.device() != device || !s.kept.is_contiguous()) refuse("the workspace must be contiguous and on " + device.str());
  }
  return s;
}

// ---------------------------------------------------------------- results
PyObject *status(svdq_status s) { return PyLong_FromLong(s); }
PyObject *wrap(const Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
PyObject *tuple(std::initializer_list<Tensor> ts) {
  PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor &t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

// ---------------------------------------------------------------- layer norm
// X, weight, bias, rows_per_group, weight_offset, eps, Y, stats
PyObject *layer_norm(PyObject *const *a) {
  const Tensor &X = tensor(a[0], "X");
  const int code = float_code(X, "X");
  const Rows r = rows_of(X, "X");
  const at::Device device = X.device();
  const svdq_norm_affine af = affine_of(X, r, a[1], a[2], integer(a[3]), number(a[4]), 0);
  const float eps = number(a[5]);
  size_t stride = 0;
  Tensor Y = output(a[6], "Y", r, X, &stride), mean, rstd;
  const bool stats = truth(a[7]);
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(device);
    if (!Y.defined()) Y = fresh({r.M, r.K}, X.scalar_type(), device);
    if (stats) {
      mean = fresh({r.M}, at::kFloat, device);
      rstd = fresh({r.M}, at::kFloat, device);
    }
    st = entry.layer_norm(X.data_ptr(), r.stride, code, r.M, r.K, &af, eps, Y.data_ptr(), stride,
                          stats ? mean.data_ptr<float>() : nullptr, stats ? rstd.data_ptr<float>() : nullptr, stream_of(device));
  }
  if (st != SVDQ_OK) return status(st);
  return stats ? tuple({Y, mean, rstd}) : wrap(Y);
}

// dY, X, mean, rstd, weight, rows_per_group, weight_offset, dX, groups, need_dX, need_dweight, need_dbias, workspace
PyObject *layer_norm_backward(PyObject *const *a) {
  const Tensor &X = tensor(a[1], "X");
  const int code = float_code(X, "X");
  const Rows r = rows_of(X, "X");
  const at::Device device = X.device();
  const Tensor &dY = tensor(a[0], "dY");
  const Rows d = rows_of(dY, "dY");
  if (d.M != r.M || d.K != r.K || dY.scalar_type() != X.scalar_type() || dY.device() != device)
    refuse("dY must have X's shape, type and device");
  const int64_t groups = has(a[8]) ? integer(a[8]) : 0;
  if (groups < 0 || (has(a[8]) && groups == 0)) refuse("no groups");
  const svdq_norm_affine af = affine_of(X, r, a[4], Py_None, integer(a[5]), number(a[6]), groups);
  if (!has(a[2]) || !has(a[3])) refuse("mean and rstd must be given");
  const float *mean = floats(a[2], "mean", r.M, device), *rstd = floats(a[3], "rstd", r.M, device);
  const bool need_dX = truth(a[9]), need_dw = truth(a[10]), need_db = truth(a[11]);
  size_t stride = static_cast<size_t>(r.K);
  Tensor dX, dw, db;
  if (need_dX) dX = output(a[7], "dX", r, X, &stride);
  Space s = space_of(a[12], device);
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(device);
    if (need_dX && !dX.defined()) dX = fresh({r.M, r.K}, X.scalar_type(), device);
    if (need_dw) dw = fresh({af.groups, r.K}, at::kFloat, device);
    if (need_db) db = fresh({af.groups, r.K}, at::kFloat, device);
    s.make(need_dw || need_db ? entry.layer_norm_workspace_bytes(r.M, r.K, af.groups, af.rows_per_group) : 0, device);
    st = entry.layer_norm_backward(dY.data_ptr(), d.stride, X.data_ptr(), r.stride, code, r.M, r.K, &af, mean, rstd,
                                   need_dX ? dX.data_ptr() : nullptr, stride, need_dw ? dw.data_ptr<float>() : nullptr,
                                   need_db ? db.data_ptr<float>() : nullptr, s.data, s.bytes, stream_of(device));
  }
  return st != SVDQ_OK ? status(st) : tuple({dX, dw, db});
}

// ---------------------------------------------------------------- 8-bit linear
// Int8 rows and their scales: the caller's or new ones.
struct I8Rows {
  Tensor xq, scale;
  int8_t *q = nullptr;
  float *s = nullptr;

  void make(const Rows &r, const at::Device &device) {
    if (!xq.defined()) xq = fresh({r.M, r.K}, at::kChar, device);
    if (!scale.defined()) scale = fresh({r.M}, at::kFloat, device);
    q = static_cast<int8_t *>(xq.data_ptr());
    s = static_cast<float *>(scale.data_ptr());
  }
};
I8Rows i8_rows(PyObject *xq, PyObject *scale, const Rows &r, const at::Device &device) {
  I8Rows o;
  if (has(xq)) {
    values(xq, "xq", static_cast<int64_t>(r.M) * r.K, at::kChar, device);
    o.xq = tensor(xq, "xq");
  }
  if (has(scale)) {
    values(scale, "x_scale", r.M, at::kFloat, device);
    o.scale = tensor(scale, "x_scale");
  }
  return o;
}

// X, col_scale, xq, x_scale
PyObject *i8_quantize_rows(PyObject *const *a) {
  const Tensor &X = tensor(a[0], "X");
  const int code = float_code(X, "X");
  const Rows r = rows_of(X, "X");
  const at::Device device = X.device();
  const float *col = floats(a[1], "col_scale", r.K, device);
  I8Rows o = i8_rows(a[2], a[3], r, device);
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(device);
    o.make(r, device);
    st = entry.i8_quantize_rows(X.data_ptr(), r.stride, code, r.M, r.K, col, o.q, o.s, stream_of(device));
  }
  return st != SVDQ_OK ? status(st) : tuple({o.xq, o.scale});
}

// X, weight, bias, rows_per_group, weight_offset, eps, xq, x_scale
PyObject *i8_layer_norm_quantize(PyObject *const *a) {
  const Tensor &X = tensor(a[0], "X");
  const int code = float_code(X, "X");
  const Rows r = rows_of(X, "X");
  const at::Device device = X.device();
  const svdq_norm_affine af = affine_of(X, r, a[1], a[2], integer(a[3]), number(a[4]), 0);
  const float eps = number(a[5]);
  I8Rows o = i8_rows(a[6], a[7], r, device);
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(device);
    o.make(r, device);
    st = entry.i8_layer_norm_quantize(X.data_ptr(), r.stride, code, r.M, r.K, &af, eps, o.q, o.s, stream_of(device));
  }
  return st != SVDQ_OK ? status(st) : tuple({o.xq, o.scale});
}

struct I8Weight {
  int N;
  const int8_t *wq;
  const float *scale, *bias;
};
I8Weight i8_weight(PyObject *wq, PyObject *scale, PyObject *bias, int K, const at::Device &device) {
  const Tensor &w = tensor(wq, "wq");
  if (w.dim() != 2 || w.size(1) != K) refuse("wq must be a matrix of " + std::to_string(K) + " columns");
  I8Weight o;
  o.N = count(w.size(0), "wq's rows");
  o.wq = static_cast<const int8_t *>(values(wq, "wq", w.numel(), at::kChar, device));
  if (!has(scale)) refuse("w_scale must be given");
  o.scale = floats(scale, "w_scale", o.N, device);
  o.bias = floats(bias, "bias", o.N, device);
  return o;
}
// A caller's product, or none.
Tensor i8_output(PyObject *o, int M, int N, at::ScalarType type, const at::Device &device) {
  if (!has(o)) return {};
  values(o, "Y", static_cast<int64_t>(M) * N, type, device);
  return tensor(o, "Y");
}

// xq, x_scale, wq, w_scale, bias, Y, type (svdq_dtype), workspace
PyObject *i8_gemm(PyObject *const *a) {
  const Tensor &xq = tensor(a[0], "xq");
  const Rows r = rows_of(xq, "xq");
  const at::Device device = xq.device();
  const int8_t *x = static_cast<const int8_t *>(values(a[0], "xq", xq.numel(), at::kChar, device));
  if (!has(a[1])) refuse("x_scale must be given");
  const float *xs = floats(a[1], "x_scale", r.M, device);
  const I8Weight w = i8_weight(a[2], a[3], a[4], r.K, device);
  const int code = static_cast<int>(integer(a[6]));
  const at::ScalarType type = code == SVDQ_BF16 ? at::kBFloat16 : (code == SVDQ_F16 ? at::kHalf : at::kFloat);
  Tensor Y = i8_output(a[5], r.M, w.N, type, device);
  Space s = space_of(a[7], device);
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(device);
    if (!Y.defined()) Y = fresh({r.M, w.N}, type, device);
    s.make(entry.i8_workspace_bytes(r.M, w.N, r.K), device);
    st = entry.i8_gemm(x, xs, r.M, w.wq, w.scale, w.bias, w.N, r.K, Y.data_ptr(), code, s.data, s.bytes, stream_of(device));
  }
  return st != SVDQ_OK ? status(st) : wrap(Y);
}

// X, wq, w_scale, bias, col_scale, xq, x_scale, Y, workspace
PyObject *i8_linear_forward(PyObject *const *a) {
  const Tensor &X = tensor(a[0], "X");
  const int code = float_code(X, "X");
  const Rows r = rows_of(X, "X");
  const at::Device device = X.device();
  const I8Weight w = i8_weight(a[1], a[2], a[3], r.K, device);
  const float *col = floats(a[4], "col_scale", r.K, device);
  Tensor Y = i8_output(a[7], r.M, w.N, X.scalar_type(), device);
  const bool scratch = !has(a[5]) && !has(a[6]) && !has(a[8]);
  I8Rows x = i8_rows(a[5], a[6], r, device);
  Space s = space_of(a[8], device);
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(device);
    if (!Y.defined()) Y = fresh({r.M, w.N}, X.scalar_type(), device);
    const size_t need = entry.i8_workspace_bytes(r.M, w.N, r.K);
    if (scratch) {
      // scratch in one piece: the rows (16-byte multiples, or the library refuses K), the workspace, the scales
      const size_t n = (static_cast<size_t>(r.M) * r.K + 15) / 16 * 16;
      s.kept = fresh({static_cast<int64_t>(n + need + 4 * static_cast<size_t>(r.M))}, at::kChar, device);
      x.q = static_cast<int8_t *>(s.kept.data_ptr());
      x.s = reinterpret_cast<float *>(x.q + n + need);
      s.data = need ? x.q + n : nullptr;
      s.bytes = need;
    } else {
      x.make(r, device);
      s.make(need, device);
    }
    st = entry.i8_linear_forward(X.data_ptr(), r.stride, code, r.M, col, w.wq, w.scale, w.bias, w.N, r.K, x.q, x.s, Y.data_ptr(),
                                 s.data, s.bytes, stream_of(device));
  }
  return st != SVDQ_OK ? status(st) : wrap(Y);
}

// ---------------------------------------------------------------- rotary positions
const svdq_rope_axes *axes_of(PyObject *o) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != static_cast<Py_ssize_t>(sizeof(svdq_rope_axes))) refuse("axes must be a RopeAxes");
  return reinterpret_cast<const svdq_rope_axes *>(PyBytes_AS_STRING(o));
}

svdq_positions positions_of(const Tensor &pos, const svdq_rope_axes &ax) {
  svdq_positions p{};
  p.dtype = dtype_code(pos.scalar_type());
  if (p.dtype < SVDQ_F32) refuse("pos must be of int32, int64 or fp32");
  const int64_t d = pos.dim();
  if (d < 1 || d > 2 || (d == 2 ? pos.size(1) : 1) != ax.n_axes) refuse("pos must be [tokens, " + std::to_string(ax.n_axes) + "]");
  p.data = pos.data_ptr();
  p.token_stride = static_cast<size_t>(pos.stride(0));
  p.axis_stride = d == 2 ? static_cast<size_t>(pos.stride(1)) : 0;
  return p;
}

// pos, axes, table
PyObject *rope_axes_table(PyObject *const *a) {
  const Tensor &pos = tensor(a[0], "pos");
  const svdq_rope_axes *ax = axes_of(a[1]);
  const svdq_positions p = positions_of(pos, *ax);
  const int M = count(pos.size(0), "tokens");
  int64_t P = 0;
  for (int i = 0; i < ax->n_axes && i < 4; ++i) P += ax->pairs[i];
  Tensor table;
  if (has(a[2])) {
    values(a[2], "table", 2 * P * M, at::kFloat, pos.device());
    table = tensor(a[2], "table");
  }
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(pos.device());
    if (!table.defined()) table = fresh({M, P, 2}, at::kFloat, pos.device());
    st = entry.rope_axes_table(&p, M, ax, static_cast<float *>(table.data_ptr()), stream_of(pos.device()));
  }
  return st != SVDQ_OK ? status(st) : wrap(table);
}

// Heads [M, H, D] and their output: the caller's or a new one.
struct Heads {
  svdq_heads in{}, out{};
  Tensor kept;

  void make(const Tensor &t) {
    if (!kept.defined()) kept = fresh(t.sizes(), t.scalar_type(), t.device());
    out = {kept.data_ptr(), in.heads, static_cast<size_t>(kept.stride(0)), static_cast<size_t>(kept.stride(1))};
  }
};
Heads heads_of(const Tensor &t, PyObject *o, const char *name, const Tensor &like) {
  if (t.dim() != 3 || t.scalar_type() != like.scalar_type() || t.device() != like.device() || t.size(0) != like.size(0) ||
      t.size(2) != like.size(2))
    refuse(std::string(name) + " must be [tokens, heads, columns] like q, of its type and on its device");
  Heads h;
  if (has(o)) {
    const Tensor &u = tensor(o, "output");
    if (u.dim() != 3 || u.sizes() != t.sizes() || u.scalar_type() != t.scalar_type() || u.device() != t.device())
      refuse(std::string(name) + "_out must be like " + name);
    h.kept = u;
  }
  if (t.size(2) > 1 && (t.stride(2) != 1 || (has(o) && h.kept.stride(2) != 1)))
    refuse("the columns of " + std::string(name) + " and its output must be contiguous");
  h.in = {t.data_ptr(), count(t.size(1), "heads"), static_cast<size_t>(t.stride(0)), static_cast<size_t>(t.stride(1))};
  return h;
}

// q, k, pos, axes, inverse, q_out, k_out
PyObject *rope_axes_apply(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q");
  const int code = float_code(q, "q");
  if (q.dim() != 3) refuse("q must be [tokens, heads, columns]");
  const Tensor &pos = tensor(a[2], "pos");
  const svdq_rope_axes *ax = axes_of(a[3]);
  const svdq_positions p = positions_of(pos, *ax);
  if (pos.size(0) != q.size(0) || pos.device() != q.device()) refuse("pos must have q's tokens and device");
  const int M = count(q.size(0), "tokens"), D = count(q.size(2), "columns"), inverse = truth(a[4]) ? 1 : 0;
  Heads hq = heads_of(q, a[5], "q", q), hk;
  const Tensor *k = has(a[1]) ? &tensor(a[1], "k") : nullptr;
  if (k) hk = heads_of(*k, a[6], "k", q);
  svdq_status st;
  {
    const Unlocked unlocked;
    const c10::cuda::CUDAGuard guard(q.device());
    hq.make(q);
    if (k) hk.make(*k);
    st = entry.rope_axes_apply(&hq.in, &hq.out, k ? &hk.in : nullptr, k ? &hk.out : nullptr, code, M, D, &p, ax, inverse,
                               stream_of(q.device()));
  }
  return st != SVDQ_OK ? status(st) : tuple({hq.kept, hk.kept});
}

// ---------------------------------------------------------------- module
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", N, static_cast<int>(n));
    return nullptr;
  }
  if (!entry.rope_axes_apply) {
    PyErr_SetString(PyExc_RuntimeError, "the library has not been loaded");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// The entry points' addresses, in the order of Entry.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void **to = reinterpret_cast<void **>(&entry);
  if (n != static_cast<Py_ssize_t>(sizeof(Entry) / sizeof(void *))) {
    PyErr_SetString(PyExc_TypeError, "one address for each entry point expected");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    void *p = PyLong_AsVoidPtr(args[i]);
    if (!p && PyErr_Occurred()) return nullptr;
    to[i] = p;
  }
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"layer_norm", fast(call<layer_norm, 8>), METH_FASTCALL, nullptr},
    {"layer_norm_backward", fast(call<layer_norm_backward, 13>), METH_FASTCALL, nullptr},
    {"i8_quantize_rows", fast(call<i8_quantize_rows, 4>), METH_FASTCALL, nullptr},
    {"i8_layer_norm_quantize", fast(call<i8_layer_norm_quantize, 8>), METH_FASTCALL, nullptr},
    {"i8_gemm", fast(call<i8_gemm, 8>), METH_FASTCALL, nullptr},
    {"i8_linear_forward", fast(call<i8_linear_forward, 9>), METH_FASTCALL, nullptr},
    {"rope_axes_table", fast(call<rope_axes_table, 3>), METH_FASTCALL, nullptr},
    {"rope_axes_apply", fast(call<rope_axes_apply, 7>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
