// Tensors to descriptors for the layer entry points, as a CPython module.
//
// A short layer call takes the GPU 2 to 7 us, less than Python needs to look at a dozen
// tensors (13 to 26 us a call through ctypes), so the checks, the allocations and the call
// of the C ABI happen here.  The functions take their arguments by position;
// newton_schulz_11_b200/layers.py has the signatures, the documentation and the streams.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "muon_b200.h"

namespace {

struct Refused {
  PyObject* type;
  std::string text;
};

[[noreturn]] void refuse(PyObject* type, const std::string& text) { throw Refused{type, text}; }

std::string shape_text(at::IntArrayRef s) {
  std::string o = "(";
  for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
  return o + (s.size() == 1 ? ",)" : ")");
}

std::string dtype_text(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "float32";
    case at::kBFloat16: return "bfloat16";
    case at::kHalf: return "float16";
    case at::kDouble: return "float64";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(what) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// The call's first matrix: 2-D, on a GPU.
const at::Tensor& first(PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 2)
    refuse(PyExc_ValueError, std::string(what) + " must be 2-D, got shape " + shape_text(t.sizes()));
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(what) + " must live on a CUDA device");
  return t;
}

constexpr at::ScalarType kAny = at::ScalarType::Undefined;

int32_t dtype_code(const at::Tensor& t, const char* what, at::ScalarType want) {
  const at::ScalarType d = t.scalar_type();
  if ((d != at::kFloat && d != at::kBFloat16) || (want != kAny && d != want))
    refuse(PyExc_TypeError, std::string(what) + " has dtype " + dtype_text(d) + ", expected " +
                                (want == kAny ? "float32 or bfloat16" : dtype_text(want)));
  return d == at::kBFloat16 ? MUON_BF16 : MUON_F32;
}

void check_device(const at::Tensor& t, const char* what, c10::Device device) {
  if (t.device() != device)
    refuse(PyExc_ValueError, std::string(what) + " is on " + t.device().str() + ", expected " + device.str());
}

muon_view_t matrix(const at::Tensor& t, const char* what, int64_t rows, int64_t cols, c10::Device device,
                   at::ScalarType want = kAny) {
  muon_view_t v{nullptr, cols, dtype_code(t, what, want), 0};
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(PyExc_ValueError, std::string(what) + " has shape " + shape_text(t.sizes()) + ", expected " +
                                 shape_text({rows, cols}));
  check_device(t, what, device);
  if (t.stride(1) != 1 && cols > 1 && rows > 0)
    refuse(PyExc_ValueError, std::string(what) + " must have unit stride along its last dimension");
  if (rows > 1) {
    v.ld = t.stride(0);
    if (v.ld < cols)
      refuse(PyExc_ValueError, std::string(what) + " must not repeat rows (stride " + std::to_string(v.ld) + " for " +
                                   std::to_string(cols) + " columns)");
  }
  v.data = t.data_ptr();
  return v;
}

muon_view_t vector(const at::Tensor& t, const char* what, int64_t n, c10::Device device, at::ScalarType want = kAny) {
  muon_view_t v{nullptr, n, dtype_code(t, what, want), 0};
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(what) + " must be a contiguous vector of " + std::to_string(n) +
                                 " elements, got shape " + shape_text(t.sizes()));
  check_device(t, what, device);
  v.data = t.data_ptr();
  return v;
}

bool given(PyObject* o) { return o != Py_None; }

muon_view_t matrix_or_absent(PyObject* o, const char* what, int64_t rows, int64_t cols, c10::Device device) {
  return given(o) ? matrix(tensor(o, what), what, rows, cols, device) : muon_view_t{nullptr, 0, 0, 0};
}

muon_view_t vector_or_absent(PyObject* o, const char* what, int64_t n, c10::Device device) {
  return given(o) ? vector(tensor(o, what), what, n, device) : muon_view_t{nullptr, 0, 0, 0};
}

at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType dtype, c10::Device device) {
  return at::detail::empty_cuda(sizes, dtype, device, c10::nullopt);
}

// The tensor given, or a new one.
at::Tensor output(PyObject* o, const char* what, at::IntArrayRef sizes, at::ScalarType dtype, c10::Device device) {
  return given(o) ? tensor(o, what) : fresh(sizes, dtype, device);
}

float* f32_vector(const at::Tensor& t, const char* what, int64_t n, c10::Device device) {
  return static_cast<float*>(vector(t, what, n, device, at::kFloat).data);
}

// A call that the C ABI refused becomes the package's MuonError.
PyObject* g_error = nullptr;

void check(muon_status_t st, const char* where) {
  if (st == MUON_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(st), where);
  if (e != nullptr) {
    PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
    Py_DECREF(e);
  }
  throw python_error();
}

// A new reference that is dropped at the end of the scope.
struct Held {
  PyObject* o;
  explicit Held(PyObject* p) : o(p) {}
  ~Held() { Py_XDECREF(o); }
  Held(const Held&) = delete;
};

// A Workspace on another device would hand its memory to kernels on this one.
void check_workspace(PyObject* w, c10::Device device) {
  const Held on(PyObject_GetAttrString(w, "device")), buf(PyObject_GetAttrString(w, "buf"));
  if (on.o == nullptr || buf.o == nullptr || !THPDevice_Check(on.o)) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "workspace must be a Workspace");
  }
  c10::Device at = reinterpret_cast<THPDevice*>(on.o)->device;  // without an index: where its buffer is, if it has one
  if (THPVariable_Check(buf.o)) at = THPVariable_Unpack(buf.o).device();
  if (at.type() != device.type() || (at.has_index() && at.index() != device.index()))
    refuse(PyExc_ValueError, "workspace is on " + at.str() + ", expected " + device.str());
}

// The call's scratch: from the caller's Workspace, or from the allocator on this stream.
struct Scratch {
  void* ptr = nullptr;
  size_t bytes = 0;
  at::Tensor buf;

  Scratch(size_t need, PyObject* workspace, c10::Device device, void* stream) : bytes(need) {
    if (given(workspace)) check_workspace(workspace, device);
    if (need == 0) return;
    if (given(workspace)) {
      PyObject* r = PyObject_CallMethod(workspace, "ensure", "nK", static_cast<Py_ssize_t>(need),
                                        reinterpret_cast<unsigned long long>(stream));
      if (r == nullptr) throw python_error();
      PyObject* p = PyTuple_Check(r) && PyTuple_GET_SIZE(r) == 2 ? PyTuple_GET_ITEM(r, 0) : nullptr;
      ptr = p != nullptr ? PyLong_AsVoidPtr(p) : nullptr;
      Py_DECREF(r);
      if (ptr == nullptr) refuse(PyExc_TypeError, "workspace must be a Workspace");
    } else {
      buf = fresh({static_cast<int64_t>(need)}, at::kByte, device);
      ptr = buf.data_ptr();
    }
  }
};

void* current_stream(c10::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

PyObject* wrap_or_none(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

PyObject* pack3(const at::Tensor& a, const at::Tensor& b, const at::Tensor& c) {
  PyObject* r = PyTuple_New(3);
  if (r == nullptr) throw python_error();
  const at::Tensor* t[3] = {&a, &b, &c};
  for (int i = 0; i < 3; ++i) {
    PyObject* o = wrap_or_none(*t[i]);
    if (o == nullptr) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return static_cast<int>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// (x, gain, bias, eps, out) -> (y, mean, rstd)
PyObject* layer_norm(PyObject* const* a) {
  const at::Tensor& x = first(a[0], "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  const c10::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  muon_layer_norm_t d{};
  d.x = matrix(x, "x", rows, cols, device);
  d.gain = vector_or_absent(a[1], "gain", cols, device);
  d.bias = vector_or_absent(a[2], "bias", cols, device);
  const at::Tensor y = output(a[4], "out", {rows, cols}, x.scalar_type(), device);
  d.y = matrix(y, "out", rows, cols, device, x.scalar_type());
  const at::Tensor mean = fresh({rows}, at::kFloat, device), rstd = fresh({rows}, at::kFloat, device);
  d.mean = static_cast<float*>(mean.data_ptr());
  d.rstd = static_cast<float*>(rstd.data_ptr());
  d.rows = rows;
  d.cols = cols;
  d.eps = static_cast<float>(eps);
  check(muon_layer_norm(&d, current_stream(device)), "muon_layer_norm");
  return pack3(y, mean, rstd);
}

// (dy, x, mean, rstd, gain, skip, dx, dgain, dbias, need_dx, need_dgain, need_dbias, accumulate, workspace)
// -> (dx, dgain, dbias)
PyObject* layer_norm_backward(PyObject* const* a) {
  const at::Tensor& x = first(a[1], "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  const c10::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const bool need_dx = truth(a[9]), need_dgain = truth(a[10]), need_dbias = truth(a[11]);
  muon_layer_norm_grad_t d{};
  d.accumulate = truth(a[12]) ? 1 : 0;
  if (d.accumulate && ((need_dgain && !given(a[7])) || (need_dbias && !given(a[8]))))
    refuse(PyExc_ValueError, "accumulate needs dgain and dbias");
  if (!(need_dx || need_dgain || need_dbias)) refuse(PyExc_ValueError, "nothing to compute");
  const at::ScalarType xt = x.scalar_type();
  d.x = matrix(x, "x", rows, cols, device);
  d.dy = matrix(tensor(a[0], "dy"), "dy", rows, cols, device, xt);
  d.mean = f32_vector(tensor(a[2], "mean"), "mean", rows, device);
  d.rstd = f32_vector(tensor(a[3], "rstd"), "rstd", rows, device);
  d.gain = vector_or_absent(a[4], "gain", cols, device);
  at::Tensor dx, dgain, dbias;
  if (need_dx) {
    dx = output(a[6], "dx", {rows, cols}, xt, device);
    d.dx = matrix(dx, "dx", rows, cols, device, xt);
    d.skip = matrix_or_absent(a[5], "skip", rows, cols, device);
  }
  if (need_dgain) {
    dgain = output(a[7], "dgain", {cols}, at::kFloat, device);
    d.dgain = f32_vector(dgain, "dgain", cols, device);
  }
  if (need_dbias) {
    dbias = output(a[8], "dbias", {cols}, at::kFloat, device);
    d.dbias = f32_vector(dbias, "dbias", cols, device);
  }
  d.rows = rows;
  d.cols = cols;
  void* stream = current_stream(device);
  size_t need = 0;
  check(muon_layer_norm_backward_workspace(&d, &need), "muon_layer_norm_backward");
  const Scratch ws(need, a[13], device, stream);
  check(muon_layer_norm_backward(&d, ws.ptr, ws.bytes, stream), "muon_layer_norm_backward");
  return pack3(dx, dgain, dbias);
}

// (x, w, bias, act, residual, out, save_preact, preact, workspace) -> y or (y, z)
PyObject* linear(PyObject* const* a) {
  const at::Tensor& x = first(a[0], "x");
  const at::Tensor& w = first(a[1], "w");
  const int64_t rows = x.size(0), in = x.size(1), out = w.size(0);
  const c10::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  muon_linear_t d{};
  d.act = as_int(a[3]);
  d.x = matrix(x, "x", rows, in, device);
  d.w = matrix(w, "w", out, in, device);
  d.bias = vector_or_absent(a[2], "bias", out, device);
  d.residual = matrix_or_absent(a[4], "residual", rows, out, device);
  const at::Tensor y = output(a[5], "out", {rows, out}, x.scalar_type(), device);
  d.y = matrix(y, "out", rows, out, device);
  at::Tensor z;
  if (given(a[7]) || truth(a[6])) {
    z = output(a[7], "preact", {rows, out}, x.scalar_type(), device);
    d.preact = matrix(z, "preact", rows, out, device);
  }
  d.rows = rows;
  d.in = in;
  d.out = out;
  void* stream = current_stream(device);
  size_t need = 0;
  check(muon_linear_workspace(&d, &need), "muon_linear");
  const Scratch ws(need, a[8], device, stream);
  check(muon_linear(&d, ws.ptr, ws.bytes, stream), "muon_linear");
  if (!z.defined()) return THPVariable_Wrap(y);
  PyObject *py = THPVariable_Wrap(y), *pz = py == nullptr ? nullptr : THPVariable_Wrap(z);
  PyObject* r = pz == nullptr ? nullptr : PyTuple_Pack(2, py, pz);
  Py_XDECREF(py);
  Py_XDECREF(pz);
  return r;
}

// (dy, x, w, in_act, in_preact, skip, dx, dw, db, need_dx, need_dw, need_db, accumulate, workspace)
// -> (dx, dw, db)
PyObject* linear_backward(PyObject* const* a) {
  const at::Tensor& dy = first(a[0], "dy");
  const at::Tensor& w = first(a[2], "w");
  const int64_t rows = dy.size(0), out = dy.size(1), in = w.size(1);
  const c10::Device device = dy.device();
  const c10::cuda::CUDAGuard guard(device);
  const bool need_dx = truth(a[9]), need_dw = truth(a[10]), need_db = truth(a[11]);
  muon_linear_grad_t d{};
  d.in_act = as_int(a[3]);
  d.accumulate = truth(a[12]) ? 1 : 0;
  if (d.in_act != MUON_ACT_NONE && need_dx && !given(a[4])) refuse(PyExc_ValueError, "in_act needs in_preact");
  if (d.accumulate && ((need_dw && !given(a[7])) || (need_db && !given(a[8]))))
    refuse(PyExc_ValueError, "accumulate needs dw and db");
  if (!(need_dx || need_dw || need_db)) refuse(PyExc_ValueError, "nothing to compute");
  d.dy = matrix(dy, "dy", rows, out, device);
  d.x = matrix(tensor(a[1], "x"), "x", rows, in, device);
  d.w = matrix(w, "w", out, in, device);
  if (d.in_act != MUON_ACT_NONE) d.preact = matrix_or_absent(a[4], "in_preact", rows, in, device);
  at::Tensor dx, dw, db;
  if (need_dx) {
    dx = output(a[6], "dx", {rows, in}, dy.scalar_type(), device);
    d.dx = matrix(dx, "dx", rows, in, device);
    d.skip = matrix_or_absent(a[5], "skip", rows, in, device);
  }
  if (need_dw) {
    dw = output(a[7], "dw", {out, in}, at::kFloat, device);
    d.dw = matrix(dw, "dw", out, in, device, at::kFloat);
  }
  if (need_db) {
    db = output(a[8], "db", {out}, at::kFloat, device);
    d.db = f32_vector(db, "db", out, device);
  }
  d.rows = rows;
  d.in = in;
  d.out = out;
  void* stream = current_stream(device);
  size_t need = 0;
  check(muon_linear_backward_workspace(&d, &need), "muon_linear_backward");
  const Scratch ws(need, a[13], device, stream);
  check(muon_linear_backward(&d, ws.ptr, ws.bytes, stream), "muon_linear_backward");
  return pack3(dx, dw, db);
}

// (dy, preact, act, out) -> dz
PyObject* activation_backward(PyObject* const* a) {
  const at::Tensor& dy = first(a[0], "dy");
  const int64_t rows = dy.size(0), cols = dy.size(1);
  const c10::Device device = dy.device();
  const c10::cuda::CUDAGuard guard(device);
  muon_activation_grad_t d{};
  d.act = as_int(a[2]);
  if (d.act == MUON_ACT_NONE) refuse(PyExc_ValueError, "act must name an activation");
  d.dy = matrix(dy, "dy", rows, cols, device);
  d.z = matrix(tensor(a[1], "preact"), "preact", rows, cols, device);
  const at::Tensor dz = output(a[3], "out", {rows, cols}, dy.scalar_type(), device);
  d.dz = matrix(dz, "out", rows, cols, device, dy.scalar_type());
  d.rows = rows;
  d.cols = cols;
  check(muon_activation_backward(&d, current_stream(device)), "muon_activation_backward");
  return THPVariable_Wrap(dz);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<layer_norm, 5>("layer_norm"),
    method<layer_norm_backward, 14>("layer_norm_backward"),
    method<linear, 9>("linear"),
    method<linear_backward, 14>("linear_backward"),
    method<activation_backward, 4>("activation_backward"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers() { return PyModule_Create(&g_module); }
