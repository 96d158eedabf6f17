// Marshalling of the operators beside the scan for torch: a CPython module
// (_ssm_torch) that checks tensors, allocates outputs and scratch with torch
// and calls the C ABI of include/ssm_scan.h.  A single-token step runs a few
// microseconds on the GPU; checking its dozen tensors and filling its struct
// from Python took 5 to 8 us of CPU time beside the launch's 4, here about 1.
//
// Host code only.  The entry points of the HIP library come in as addresses
// (bind), so this module loads no library by itself, and a missing library is
// reported where it always was.  Errors are Python exceptions: TypeError and
// ValueError for what a tensor is, the package's own error for a status code,
// torch's own for what torch reports.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <exception>
#include <sstream>
#include <stdexcept>
#include <string>

#include "ssm_scan.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

struct Entry {
  decltype(&ssm_selective_scan_step) scan_step;
  decltype(&ssm_causal_conv_step) conv_step;
  decltype(&ssm_causal_conv_fwd) conv_fwd;
  decltype(&ssm_causal_conv_bwd) conv_bwd;
  decltype(&ssm_causal_conv_bwd_workspace_bytes) conv_bwd_bytes;
  decltype(&ssm_layer_norm_fwd) norm_fwd;
  decltype(&ssm_layer_norm_bwd) norm_bwd;
  decltype(&ssm_layer_norm_bwd_workspace_bytes) norm_bwd_bytes;
};

Entry entry;
PyObject* handle_for = nullptr;  // device index -> handle, as an integer
PyObject* scan_error = nullptr;  // class of (code, what)
std::array<ssm_scan_t, 64> handles{};  // of the devices seen so far (handles live until the process ends)

struct TypeRefused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct ValueRefused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python exception is set

// ---- arguments -------------------------------------------------------------

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) throw TypeRefused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// A weight's number of taps, [dim, width]; one that no kernel has stays so in
// 32 bits.
int32_t taps(const Tensor& w) {
  if (w.dim() != 2 || w.size(1) < 1) throw ValueRefused("weight must be [dim, width]");
  return static_cast<int32_t>(w.size(1) < 1000 ? w.size(1) : 1000);
}

bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

int32_t io_of(const char* name, const Tensor& t) {
  if (!t.is_cuda()) throw ValueRefused("tensors must be on a GPU device");
  if (t.scalar_type() == at::kBFloat16) return SSM_IO_BF16;
  if (t.scalar_type() == at::kFloat) return SSM_IO_F32;
  throw TypeRefused(std::string(name) + " must be float32 or bfloat16");
}

void want_dims(const Tensor& t, int64_t dims, const char* what) {
  if (t.dim() != dims) throw ValueRefused(what);
}

void want_like(const char* name, const Tensor& t, Shape shape, at::ScalarType dtype, const at::Device& dev) {
  if (t.sizes() == shape && t.scalar_type() == dtype && t.device() == dev && t.layout() == at::kStrided) return;
  std::ostringstream s;
  s << name << " must be " << shape << ' ' << dtype << " on " << dev << ", got " << t.sizes() << ' ' << t.scalar_type()
    << " on " << t.device();
  throw ValueRefused(s.str());
}

// A contiguous tensor of this shape, type and device.
void dense(const char* name, const Tensor& t, Shape shape, at::ScalarType dtype, const at::Device& dev) {
  want_like(name, t, shape, dtype, dev);
  if (!t.is_contiguous()) throw ValueRefused(std::string(name) + " must be contiguous");
}

// One whose last dimension is dense; the other strides go to the library.
void rows(const char* name, const Tensor& t, Shape shape, at::ScalarType dtype, const at::Device& dev) {
  want_like(name, t, shape, dtype, dev);
  if (shape.back() > 1 && t.stride(-1) != 1)
    throw ValueRefused(std::string(name) + " must have stride 1 in its last dimension");
}

// An optional dense tensor's address.
template <typename T>
const T* given(const char* name, PyObject* o, Shape shape, at::ScalarType dtype, const at::Device& dev) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(name, o);
  dense(name, t, shape, dtype, dev);
  return static_cast<const T*>(t.const_data_ptr());
}

Tensor fresh(Shape shape, at::ScalarType dtype, const at::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}

// An output: the one given, checked, or a new one.
enum class Layout { kDense, kRows };
Tensor output(const char* name, PyObject* o, Shape shape, at::ScalarType dtype, const at::Device& dev, Layout layout) {
  if (o == Py_None) return fresh(shape, dtype, dev);
  const Tensor& t = tensor(name, o);
  if (layout == Layout::kRows)
    rows(name, t, shape, dtype, dev);
  else
    dense(name, t, shape, dtype, dev);
  return t;
}

Tensor scratch(PyObject* o, int64_t bytes, const at::Device& dev) {
  if (bytes < 0) throw ValueRefused("unsupported sizes");
  if (o == Py_None) return fresh({bytes < 4 ? 4 : bytes}, at::kByte, dev);
  const Tensor& t = tensor("workspace", o);
  if (t.scalar_type() != at::kByte || t.device() != dev || !t.is_contiguous() || t.numel() < bytes) {
    std::ostringstream s;
    s << "workspace must be a contiguous uint8 tensor of at least " << bytes << " bytes on " << dev;
    throw ValueRefused(s.str());
  }
  return t;
}

template <typename T>
T* at_ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// ---- calls -----------------------------------------------------------------

ssm_scan_t handle_of(int64_t index) {
  if (index >= 0 && index < static_cast<int64_t>(handles.size()) && handles[index] != nullptr) return handles[index];
  PyObject* r = PyObject_CallFunction(handle_for, "L", static_cast<long long>(index));
  if (r == nullptr) throw Raised();
  void* h = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  if (h == nullptr && PyErr_Occurred()) throw Raised();
  if (index >= 0 && index < static_cast<int64_t>(handles.size())) handles[index] = static_cast<ssm_scan_t>(h);
  return static_cast<ssm_scan_t>(h);
}

// On the device's current stream, with the device current.
template <typename F, typename D, typename I>
void call(const char* name, F fn, const at::Device& dev, const D& dims, const I& io) {
  const c10::DeviceGuard guard(dev);
  const int rc = fn(handle_of(dev.index()), &dims, &io, c10::hip::getCurrentHIPStream(dev.index()).stream());
  if (rc == SSM_OK) return;
  PyObject* e = PyObject_CallFunction(scan_error, "is", rc, name);
  if (e != nullptr) {
    PyErr_SetObject(scan_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// The caller's own tensors that a call wrote, for torch's version counters: an
// autograd graph that saved one for its backward refuses to run, as after any
// operation in place.  (Inference tensors have no counter.)
void written(PyObject* o, const Tensor& t) {
  if (o != Py_None && t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw Raised();
  return o;
}

// A tuple of tensors (undefined ones as None).
template <size_t N>
PyObject* pack(const std::array<Tensor, N>& ts) {
  PyObject* tuple = PyTuple_New(N);
  if (tuple == nullptr) throw Raised();
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = nullptr;
    try {
      o = wrap(ts[i]);
    } catch (...) {
      Py_DECREF(tuple);
      throw;
    }
    PyTuple_SET_ITEM(tuple, i, o);
  }
  return tuple;
}

// The C++ body of a Python function, its exceptions turned into Python's.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, const F& body) {
  try {
    if (got != want) throw TypeRefused("wrong number of arguments");
    return body();
  } catch (const Raised&) {
  } catch (const TypeRefused& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const ValueRefused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {  // torch's own, as torch reports them (an allocation that fails is its OutOfMemoryError)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// ---- single tokens ---------------------------------------------------------

// A step's cache, where it goes and its slots.
struct Cache {
  Tensor from, to;
  const int32_t* slots;
  int64_t rows;
};

Cache cache(const char* name, PyObject* from, PyObject* to, PyObject* slots, int64_t batch, int64_t a, int64_t b,
            at::ScalarType dtype, const at::Device& dev) {
  Cache c;
  c.from = tensor(name, from);
  c.rows = slots == Py_None ? batch : c.from.size(0);
  const std::array<int64_t, 3> shape{c.rows, a, b};
  dense(name, c.from, shape, dtype, dev);
  c.to = to == Py_None ? c.from : tensor(name, to);
  if (!c.to.is_same(c.from)) dense((std::string(name) + "'s output").c_str(), c.to, shape, dtype, dev);
  c.slots = given<int32_t>("slots", slots, {batch}, at::kInt, dev);
  return c;
}

// x, delta, A_log, B, C, D, h, slots, h_last, softplus, clamp (None or a pair), delta_bias, z, y
PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Tensor &x = tensor("x", a[0]), &delta = tensor("delta", a[1]), &A = tensor("A_log", a[2]),
                 &B = tensor("B", a[3]), &C = tensor("C", a[4]), &h = tensor("h", a[6]);
    const int32_t io = io_of("x", x);
    want_dims(x, 2, "x must be [batch, dim]");
    if (A.dim() != 2 || h.dim() != 3) throw ValueRefused("A_log must be [dim, dstate] and h [rows, dim, dstate]");
    const at::Device dev = x.device();
    const at::ScalarType dt = x.scalar_type();
    const int64_t nb = x.size(0), nd = x.size(1), N = A.size(1);
    rows("x", x, {nb, nd}, dt, dev);
    rows("delta", delta, {nb, nd}, dt, dev);
    rows("B", B, {nb, N}, dt, dev);
    rows("C", C, {nb, N}, dt, dev);
    dense("A_log", A, {nd, N}, at::kFloat, dev);
    ssm_scan_step_io s{};
    s.D = given<float>("D", a[5], {nd}, at::kFloat, dev);
    s.delta_bias = given<float>("delta_bias", a[11], {nd}, at::kFloat, dev);
    if (a[12] != Py_None) {
      const Tensor& z = tensor("z", a[12]);
      rows("z", z, {nb, nd}, dt, dev);
      s.z = z.const_data_ptr();
      s.z_row_stride = z.stride(0);
    }
    const Cache c = cache("h", a[6], a[8], a[7], nb, nd, N, at::kFloat, dev);
    ssm_scan_dims dims{nb, 1, nd, N, io, flag(a[9]) ? 1 : 0, 0, 0.0f, 0.0f};
    if (a[10] != Py_None) {
      PyObject* pair = PySequence_Fast(a[10], "delta_clamp must be None or (min, max)");
      if (pair == nullptr) throw Raised();
      const bool two = PySequence_Fast_GET_SIZE(pair) == 2;
      try {
        if (!two) throw ValueRefused("delta_clamp must be None or (min, max)");
        dims.delta_clamp = 1;
        dims.delta_min = number(PySequence_Fast_GET_ITEM(pair, 0));
        dims.delta_max = number(PySequence_Fast_GET_ITEM(pair, 1));
      } catch (...) {
        Py_DECREF(pair);
        throw;
      }
      Py_DECREF(pair);
    }
    const Tensor y = output("y", a[13], {nb, nd}, dt, dev, Layout::kRows);
    s.x = x.const_data_ptr(), s.delta = delta.const_data_ptr(), s.A_log = static_cast<const float*>(A.const_data_ptr());
    s.B = B.const_data_ptr(), s.C = C.const_data_ptr(), s.slots = c.slots;
    s.h0 = at_ptr<float>(c.from), s.h_last = at_ptr<float>(c.to), s.y = y.data_ptr();
    s.x_row_stride = x.stride(0), s.delta_row_stride = delta.stride(0), s.B_row_stride = B.stride(0);
    s.C_row_stride = C.stride(0), s.y_row_stride = y.stride(0), s.n_slots = c.rows;
    call("ssm_selective_scan_step", entry.scan_step, dev, dims, s);
    written(a[6], c.to), written(a[13], y);
    return wrap(y);
  });
}

// x, conv, weight, bias, silu, slots, conv_last, y
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Tensor &x = tensor("x", a[0]), &conv = tensor("conv", a[1]), &w = tensor("weight", a[2]);
    const int32_t io = io_of("x", x);
    want_dims(x, 2, "x must be [batch, dim]");
    if (conv.dim() != 3) throw ValueRefused("conv must be [rows, width - 1, dim]");
    const int32_t width = taps(w);
    const at::Device dev = x.device();
    const at::ScalarType dt = x.scalar_type();
    const int64_t nb = x.size(0), nd = x.size(1), W = w.size(1);
    rows("x", x, {nb, nd}, dt, dev);
    dense("weight", w, {nd, W}, at::kFloat, dev);
    ssm_conv_step_io s{};
    s.bias = given<float>("bias", a[3], {nd}, at::kFloat, dev);
    const Cache c = cache("conv", a[1], a[6], a[5], nb, W - 1, nd, dt, dev);
    const ssm_conv_dims dims{nb, 1, nd, width, io, flag(a[4]) ? 1 : 0};
    const Tensor y = output("y", a[7], {nb, nd}, dt, dev, Layout::kRows);
    s.x = x.const_data_ptr(), s.weight = static_cast<const float*>(w.const_data_ptr()), s.slots = c.slots;
    s.conv0 = c.from.data_ptr(), s.conv_last = c.to.data_ptr(), s.y = y.data_ptr();
    s.x_row_stride = x.stride(0), s.y_row_stride = y.stride(0), s.n_slots = c.rows;
    call("ssm_causal_conv_step", entry.conv_step, dev, dims, s);
    written(a[1], c.to), written(a[7], y);
    return wrap(y);
  });
}

// ---- short causal convolution ----------------------------------------------

struct Conv {
  Tensor x, w;
  at::Device dev{at::kCUDA, 0};
  at::ScalarType dt;
  ssm_conv_dims dims;
  const float* bias;
  const int32_t* valid_len;
  const void* conv0;
};

// a: x, weight, bias, valid_len, silu, conv0
Conv conv_args(PyObject* const* a) {
  Conv c;
  c.x = tensor("x", a[0]), c.w = tensor("weight", a[1]);
  const int32_t io = io_of("x", c.x);
  want_dims(c.x, 3, "x must be [batch, L, dim]");
  const int32_t width = taps(c.w);
  c.dev = c.x.device(), c.dt = c.x.scalar_type();
  const int64_t nb = c.x.size(0), L = c.x.size(1), nd = c.x.size(2), W = c.w.size(1);
  rows("x", c.x, {nb, L, nd}, c.dt, c.dev);
  dense("weight", c.w, {nd, W}, at::kFloat, c.dev);
  c.bias = given<float>("bias", a[2], {nd}, at::kFloat, c.dev);
  c.valid_len = given<int32_t>("valid_len", a[3], {nb}, at::kInt, c.dev);
  c.conv0 = given<void>("conv0", a[5], {nb, W - 1, nd}, c.dt, c.dev);
  c.dims = ssm_conv_dims{nb, L, nd, width, io, flag(a[4]) ? 1 : 0};
  return c;
}

// x, weight, bias, valid_len, silu, conv0, y, conv_last, return_conv_last
PyObject* conv_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Conv c = conv_args(a);
    const int64_t nb = c.dims.batch, L = c.dims.seqlen, nd = c.dims.dim, W = c.w.size(1);
    const Tensor y = output("y", a[6], {nb, L, nd}, c.dt, c.dev, Layout::kRows);
    Tensor last;
    if (a[7] != Py_None || flag(a[8])) last = output("conv_last", a[7], {nb, W - 1, nd}, c.dt, c.dev, Layout::kDense);
    ssm_conv_fwd_io s{};
    s.x = c.x.const_data_ptr(), s.weight = static_cast<const float*>(c.w.const_data_ptr()), s.bias = c.bias;
    s.valid_len = c.valid_len, s.conv0 = c.conv0, s.y = y.data_ptr(), s.conv_last = at_ptr<void>(last);
    s.x_batch_stride = c.x.stride(0), s.x_time_stride = c.x.stride(1);
    s.y_batch_stride = y.stride(0), s.y_time_stride = y.stride(1);
    call("ssm_causal_conv_fwd", entry.conv_fwd, c.dev, c.dims, s);
    written(a[6], y), written(a[7], last);
    return pack<2>({y, last});
  });
}

// x, weight, bias, valid_len, silu, conv0, dy, dconv_last, dx, workspace
PyObject* conv_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Conv c = conv_args(a);
    const int64_t nb = c.dims.batch, L = c.dims.seqlen, nd = c.dims.dim, W = c.w.size(1);
    const Tensor& dy = tensor("dy", a[6]);
    rows("dy", dy, {nb, L, nd}, c.dt, c.dev);
    ssm_conv_bwd_io s{};
    s.dconv_last = given<void>("dconv_last", a[7], {nb, W - 1, nd}, c.dt, c.dev);
    const Tensor dx = output("dx", a[8], {nb, L, nd}, c.dt, c.dev, Layout::kRows);
    const Tensor dw = fresh({nd, W}, at::kFloat, c.dev);
    Tensor db, d0;
    if (a[2] != Py_None) db = fresh({nd}, at::kFloat, c.dev);
    if (a[5] != Py_None) d0 = fresh({nb, W - 1, nd}, c.dt, c.dev);
    const Tensor ws = scratch(a[9], entry.conv_bwd_bytes(&c.dims), c.dev);
    s.x = c.x.const_data_ptr(), s.weight = static_cast<const float*>(c.w.const_data_ptr()), s.bias = c.bias;
    s.valid_len = c.valid_len, s.conv0 = c.conv0, s.dy = dy.const_data_ptr();
    s.dx = dx.data_ptr(), s.dweight = at_ptr<float>(dw), s.dbias = at_ptr<float>(db), s.dconv0 = at_ptr<void>(d0);
    s.workspace = ws.data_ptr(), s.workspace_bytes = ws.numel();
    s.x_batch_stride = c.x.stride(0), s.x_time_stride = c.x.stride(1);
    s.dy_batch_stride = dy.stride(0), s.dy_time_stride = dy.stride(1);
    s.dx_batch_stride = dx.stride(0), s.dx_time_stride = dx.stride(1);
    call("ssm_causal_conv_bwd", entry.conv_bwd, c.dev, c.dims, s);
    written(a[8], dx);
    return pack<4>({dx, dw, db, d0});
  });
}

// ---- norms -----------------------------------------------------------------

struct Norm {
  at::Device dev{at::kCUDA, 0};
  at::ScalarType dt;
  Shape shape, stats;
  ssm_norm_dims dims;
  const float* w;
  const int32_t* valid_len;
};

// The rows `t` of a norm, its weight and its valid lengths.
Norm norm_args(const char* name, const Tensor& t, PyObject* weight, PyObject* valid_len) {
  Norm m;
  const int32_t io = io_of(name, t);
  if (t.dim() != 2 && t.dim() != 3) throw ValueRefused("rows must be [rows, dim] or [batch, L, dim]");
  if (valid_len != Py_None && t.dim() != 3) throw ValueRefused("valid_len needs rows laid out as [batch, L, dim]");
  m.dev = t.device(), m.dt = t.scalar_type();
  m.shape = t.sizes(), m.stats = m.shape.slice(0, m.shape.size() - 1);
  const int64_t nb = t.size(0), L = t.dim() == 2 ? 1 : t.size(1), nd = t.size(-1);
  dense(name, t, m.shape, m.dt, m.dev);
  const Tensor& w = tensor("weight", weight);
  dense("weight", w, {nd}, at::kFloat, m.dev);
  m.w = static_cast<const float*>(w.const_data_ptr());
  m.valid_len = given<int32_t>("valid_len", valid_len, {nb}, at::kInt, m.dev);
  m.dims = ssm_norm_dims{nb, L, nd, io, io, 0, 0.0f};
  return m;
}

// The type of a residual stream beside rows of type dt.
at::ScalarType residual_type(const char* name, const Tensor& t, Norm& m) {
  const at::ScalarType r = t.scalar_type();
  if (r != m.dt && r != at::kFloat) throw TypeRefused(std::string(name) + " must be float32 or of the rows' dtype");
  m.dims.residual_dtype = r == at::kFloat ? SSM_IO_F32 : SSM_IO_BF16;
  return r;
}

// x, weight, bias, valid_len, residual, eps, rms, y, residual_out, return_stats
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Tensor& x = tensor("x", a[0]);
    Norm m = norm_args("x", x, a[1], a[3]);
    m.dims.rms = flag(a[6]) ? 1 : 0;
    m.dims.eps = number(a[5]);
    ssm_norm_fwd_io s{};
    s.bias = given<float>("bias", a[2], {m.dims.dim}, at::kFloat, m.dev);
    at::ScalarType r = m.dt;
    if (a[4] != Py_None)
      r = residual_type("residual", tensor("residual", a[4]), m);
    else if (a[8] != Py_None)
      r = residual_type("residual_out", tensor("residual_out", a[8]), m);
    s.residual = given<void>("residual", a[4], m.shape, r, m.dev);
    const Tensor y = output("y", a[7], m.shape, m.dt, m.dev, Layout::kDense);
    Tensor out, mean, rstd;
    if (a[4] != Py_None || a[8] != Py_None) out = output("residual_out", a[8], m.shape, r, m.dev, Layout::kDense);
    const bool stats = flag(a[9]);
    if (stats) {
      rstd = fresh(m.stats, at::kFloat, m.dev);
      if (!m.dims.rms) mean = fresh(m.stats, at::kFloat, m.dev);
    }
    s.x = x.const_data_ptr(), s.weight = m.w, s.valid_len = m.valid_len, s.y = y.data_ptr();
    s.residual_out = at_ptr<void>(out), s.mean = at_ptr<float>(mean), s.rstd = at_ptr<float>(rstd);
    call("ssm_layer_norm_fwd", entry.norm_fwd, m.dev, m.dims, s);
    written(a[7], y), written(a[8], out);
    return stats ? pack<4>({y, out, mean, rstd}) : pack<2>({y, out});
  });
}

// dy, v, weight, mean, rstd, valid_len, dresidual_out, with_bias, with_residual, workspace
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Tensor &dy = tensor("dy", a[0]), &v = tensor("v", a[1]);
    Norm m = norm_args("dy", dy, a[2], a[5]);
    const at::ScalarType r = residual_type("v", v, m);
    dense("v", v, m.shape, r, m.dev);
    ssm_norm_bwd_io s{};
    s.mean = given<float>("mean", a[3], m.stats, at::kFloat, m.dev);
    const Tensor& rstd = tensor("rstd", a[4]);
    dense("rstd", rstd, m.stats, at::kFloat, m.dev);
    s.dresidual_out = given<void>("dresidual_out", a[6], m.shape, r, m.dev);
    m.dims.rms = a[3] == Py_None ? 1 : 0;
    m.dims.eps = 1.0f;  // it went into rstd; the library wants a positive one all the same
    const Tensor dx = fresh(m.shape, m.dt, m.dev);
    Tensor dresidual, db;
    const bool wanted = a[8] == Py_None ? a[6] != Py_None : flag(a[8]), apart = wanted && r != m.dt;
    if (apart) dresidual = fresh(m.shape, r, m.dev);
    const Tensor dw = fresh({m.dims.dim}, at::kFloat, m.dev);
    if (flag(a[7])) db = fresh({m.dims.dim}, at::kFloat, m.dev);
    const Tensor ws = scratch(a[9], entry.norm_bwd_bytes(&m.dims), m.dev);
    s.dy = dy.const_data_ptr(), s.v = v.const_data_ptr(), s.weight = m.w;
    s.rstd = static_cast<const float*>(rstd.const_data_ptr()), s.valid_len = m.valid_len;
    s.dx = dx.data_ptr(), s.dresidual = at_ptr<void>(dresidual), s.dweight = at_ptr<float>(dw);
    s.dbias = at_ptr<float>(db), s.workspace = ws.data_ptr(), s.workspace_bytes = ws.numel();
    call("ssm_layer_norm_bwd", entry.norm_bwd, m.dev, m.dims, s);
    return pack<4>({dx, wanted ? (apart ? dresidual : dx) : Tensor(), dw, db});
  });
}

// bind(addresses of Entry's functions in its order, handle_for, error class)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    void* p[8];
    for (int i = 0; i < 8; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (p[i] == nullptr) {
        if (PyErr_Occurred()) throw Raised();
        throw ValueRefused("a NULL entry point");
      }
    }
    entry.scan_step = reinterpret_cast<decltype(entry.scan_step)>(p[0]);
    entry.conv_step = reinterpret_cast<decltype(entry.conv_step)>(p[1]);
    entry.conv_fwd = reinterpret_cast<decltype(entry.conv_fwd)>(p[2]);
    entry.conv_bwd = reinterpret_cast<decltype(entry.conv_bwd)>(p[3]);
    entry.conv_bwd_bytes = reinterpret_cast<decltype(entry.conv_bwd_bytes)>(p[4]);
    entry.norm_fwd = reinterpret_cast<decltype(entry.norm_fwd)>(p[5]);
    entry.norm_bwd = reinterpret_cast<decltype(entry.norm_bwd)>(p[6]);
    entry.norm_bwd_bytes = reinterpret_cast<decltype(entry.norm_bwd_bytes)>(p[7]);
    Py_INCREF(a[8]);
    Py_XSETREF(handle_for, a[8]);
    Py_INCREF(a[9]);
    Py_XSETREF(scan_error, a[9]);
    Py_RETURN_NONE;
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),     FAST(scan_step), FAST(conv_step), FAST(conv_fwd),
                         FAST(conv_bwd), FAST(norm_fwd),  FAST(norm_bwd),  {nullptr, nullptr, 0, nullptr}};
#undef FAST

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ssm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ssm_torch() { return PyModule_Create(&module); }
