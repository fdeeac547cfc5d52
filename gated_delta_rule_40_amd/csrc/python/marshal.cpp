// marshal.cpp -- the binding's tensor checks as a CPython extension.
//
// Every call of the library checks each tensor it is given (shape, dtype,
// device, contiguity) and takes its address.  In Python that is 0.4 us a
// tensor, which for a single-token call of ten tensors is as long as the launch;
// here it is 0.1 us.  What does not fit goes back to a Python function, which
// says what is wrong.
//
// The calls of the norms, the 8-bit product and the rotary positions are native as a
// whole (a norm of one row 6.7 -> 4.1 us a call, rotary positions of 64 tokens 6.5 -> 4.0,
// a small product 5.7 -> 3.5; the library's own part is 3.3): each function here checks
// what its Python counterpart checks and calls the library, or returns None for
// anything that is not a plain call on the current device, which the Python path then
// takes or refuses.  Their signatures here are those of include/gdr.h.
#include <Python.h>

#include <stdint.h>

#include <initializer_list>

#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* refuse = nullptr;  // called with the arguments that did not fit; raises

// Whether t is a dense tensor of exactly this shape, dtype and device.
bool fits(PyObject* t, PyObject* shape, PyObject* dtype, PyObject* device) {
  if (!THPVariable_Check(t) || !PyTuple_Check(shape) || !THPDtype_Check(dtype) ||
      !THPDevice_Check(device))
    return false;
  const at::Tensor& x = THPVariable_Unpack(t);
  if (x.layout() != at::kStrided ||
      x.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type ||
      x.device() != reinterpret_cast<THPDevice*>(device)->device)
    return false;
  const auto sizes = x.sizes();
  const Py_ssize_t n = PyTuple_GET_SIZE(shape);
  if (static_cast<Py_ssize_t>(sizes.size()) != n) return false;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const long long s = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    if (s == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    if (s != sizes[i]) return false;
  }
  return x.is_contiguous();
}

PyObject* address(PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "expected (tensor, name, shape, dtype, device)");
    return nullptr;
  }
  try {
    if (fits(a[0], a[2], a[3], a[4]))
      return PyLong_FromUnsignedLongLong(
          reinterpret_cast<unsigned long long>(THPVariable_Unpack(a[0]).data_ptr()));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  if (!refuse) {
    PyErr_SetString(PyExc_ValueError, "tensor does not fit the call");
    return nullptr;
  }
  PyObject* r = PyObject_CallFunctionObjArgs(refuse, a[0], a[1], a[2], a[3], a[4], nullptr);
  if (r) {  // it has to raise
    Py_DECREF(r);
    PyErr_SetString(PyExc_ValueError, "tensor does not fit the call");
  }
  return nullptr;
}

// ptr(tensor, name, shape, dtype, device) -> address
PyObject* ptr(PyObject*, PyObject* const* a, Py_ssize_t n) { return address(a, n); }

// The same, None for None.
PyObject* opt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n > 0 && a[0] == Py_None) Py_RETURN_NONE;
  return address(a, n);
}

// ---- whole calls ------------------------------------------------------------

// The library's entry points (include/gdr.h), and torch's accessors of the current
// device and its current stream.
struct Entries {
  int (*rms_norm)(const int32_t*, int, const void*, int64_t, int, void*, int, const void*, int64_t,
                  const float*, float, void*, void*, float*, void*);
  int (*quant_rows)(const int32_t*, int, const void*, int64_t, void*, float*, void*);
  int (*matmul_fp8)(const int32_t*, int, const void*, const float*, const void*, const float*,
                    const float*, void*, void*);
  int (*rope)(const int32_t*, int, int, const void*, int64_t, const double*, float, const int32_t*,
              const int32_t*, void*, void*, void*, void*);
  PyObject *device, *stream;
};
Entries entries = {};

// bind(rms_norm, quant_rows, matmul_fp8, rope, device, stream): addresses and callables.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "expected four addresses and two callables");
    return nullptr;
  }
  void* fn[4];
  for (int i = 0; i < 4; ++i) fn[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  Py_INCREF(a[4]);
  Py_XSETREF(entries.device, a[4]);
  Py_INCREF(a[5]);
  Py_XSETREF(entries.stream, a[5]);
  entries.rms_norm = reinterpret_cast<decltype(entries.rms_norm)>(fn[0]);
  entries.quant_rows = reinterpret_cast<decltype(entries.quant_rows)>(fn[1]);
  entries.matmul_fp8 = reinterpret_cast<decltype(entries.matmul_fp8)>(fn[2]);
  entries.rope = reinterpret_cast<decltype(entries.rope)>(fn[3]);
  Py_RETURN_NONE;
}

// A call that is not plain.  Thrown before the library is called.
struct NotPlain {};
void need(bool ok) {
  if (!ok) throw NotPlain();
}

const at::Tensor& tensor(PyObject* o, int64_t dims) {
  need(THPVariable_Check(o));
  const at::Tensor& t = THPVariable_Unpack(o);
  need(t.layout() == at::kStrided && t.dim() == dims);
  return t;
}

int io_of(const at::Tensor& t) {
  need(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16);
  return t.scalar_type() == at::kBFloat16;
}

bool is_codes(const at::Tensor& t) {
  return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte;
}

int32_t size32(int64_t n) {
  need(n >= 0 && n <= INT32_MAX);
  return static_cast<int32_t>(n);
}

// The device of a call, and what it asks of the other tensors.
struct Call {
  c10::Device device;
  long index;
  explicit Call(const at::Tensor& lead) : device(lead.device()), index(lead.device().index()) {
    need(entries.device && lead.device().type() == c10::DeviceType::CUDA);
    PyObject* here = PyObject_CallNoArgs(entries.device);
    need(here);
    const long current = PyLong_AsLong(here);
    Py_DECREF(here);
    need(current == index);
  }
  // A dense tensor of this shape and type.
  void* dense(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    need(t.layout() == at::kStrided && t.scalar_type() == type && t.device() == device &&
         t.sizes().equals(c10::IntArrayRef(shape)) && t.is_contiguous());
    return t.data_ptr();
  }
  void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    need(THPVariable_Check(o));
    return dense(THPVariable_Unpack(o), type, shape);
  }
  void* dense_or_none(PyObject* o, at::ScalarType type,
                      std::initializer_list<int64_t> shape) const {
    return o == Py_None ? nullptr : dense(o, type, shape);
  }
  void* stream() const {
    PyObject* i = PyLong_FromLong(index);
    PyObject* s = i ? PyObject_CallOneArg(entries.stream, i) : nullptr;
    Py_XDECREF(i);
    need(s);
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    need(!PyErr_Occurred());
    return p;
  }
};

// Row stride of rows whose channels are contiguous.
int64_t apart(const at::Tensor& t) {
  if (t.is_contiguous()) return t.size(1);
  need(t.size(1) <= 1 || t.stride(1) == 1);
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// Runs f, which gives a status; None where it finds that the call is not plain.
template <typename F>
PyObject* plain(F f) {
  try {
    return PyLong_FromLong(f());
  } catch (const NotPlain&) {
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

struct Unlocked {  // the library call may wait for room in the queue
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// rms_norm(x, weight, y, codes, scales, residual, gate, gate_first, heads, eps)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain([&] {
    need(n == 10);
    const at::Tensor& x = tensor(a[0], 2);
    const Call call(x);
    const int io = io_of(x);
    const int64_t R = x.size(0), W = x.size(1);
    const at::ScalarType type = x.scalar_type();
    int64_t H = 1;
    if (a[8] != Py_None) {
      H = PyLong_AsLongLong(a[8]);
      need(!PyErr_Occurred());
    }
    const float* weight = nullptr;
    if (a[1] != Py_None) {
      need(THPVariable_Check(a[1]));
      const at::Tensor& w = THPVariable_Unpack(a[1]);
      const int64_t h = w.dim() == 2 ? w.size(0) : 1;
      need((w.dim() == 1 || w.dim() == 2) && h >= 1 && W % h == 0 &&
           (a[8] == Py_None || h == H));
      H = h;
      weight = static_cast<const float*>(w.dim() == 2 ? call.dense(w, at::kFloat, {H, W / H})
                                                      : call.dense(w, at::kFloat, {W}));
    }
    need(H >= 1 && W % H == 0);
    int res = 0, order = 0;
    void* residual = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& r = tensor(a[5], 2);
      res = io_of(r);
      residual = call.dense(r, r.scalar_type(), {R, W});
    }
    const void* gate = nullptr;
    int64_t gate_row = 0;
    if (a[6] != Py_None) {
      const at::Tensor& g = tensor(a[6], 2);
      need(g.sizes().equals(x.sizes()) && g.scalar_type() == type && g.device() == x.device());
      const int first = PyObject_IsTrue(a[7]);
      need(first >= 0);
      order = first ? 2 : 1;
      gate = g.data_ptr();
      gate_row = apart(g);
    }
    void* y = call.dense_or_none(a[2], type, {R, W});
    void *codes = nullptr, *scales = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor& c = tensor(a[3], 2);
      need(is_codes(c));
      codes = call.dense(c, c.scalar_type(), {R, W});
      scales = call.dense(a[4], at::kFloat, {R, (W + 127) / 128});
    } else {
      need(a[4] == Py_None);
    }
    const double eps = PyFloat_AsDouble(a[9]);
    need(!PyErr_Occurred());
    const int32_t dims[3] = {size32(R), size32(H), size32(W / H)};
    const void* xp = x.data_ptr();
    const int64_t row = apart(x);
    void* stream = call.stream();
    Unlocked unlocked;
    return entries.rms_norm(dims, io, xp, row, res, residual, order, gate, gate_row, weight,
                            static_cast<float>(eps), y, codes, static_cast<float*>(scales),
                            stream);
  });
}

// quant_rows(x, codes, scales)
PyObject* quant_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain([&] {
    need(n == 3);
    const at::Tensor& x = tensor(a[0], 2);
    const Call call(x);
    const int io = io_of(x);
    const int64_t R = x.size(0), W = x.size(1);
    const at::Tensor& c = tensor(a[1], 2);
    need(is_codes(c) && W > 0);
    void* codes = call.dense(c, c.scalar_type(), {R, W});
    void* scales = call.dense(a[2], at::kFloat, {R, (W + 127) / 128});
    // Rows of whole blocks are heads of 128 channels side by side.
    const int64_t H = W % 128 == 0 ? W / 128 : 1;
    const int32_t dims[3] = {size32(R), size32(H), size32(W / H)};
    const void* xp = x.data_ptr();
    const int64_t row = apart(x);
    void* stream = call.stream();
    Unlocked unlocked;
    return entries.quant_rows(dims, io, xp, row, codes, static_cast<float*>(scales), stream);
  });
}

// matmul_fp8(x, x_scales, w, w_scales, y, bias)
PyObject* matmul_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain([&] {
    need(n == 6);
    const at::Tensor &y = tensor(a[4], 2), &x = tensor(a[0], 2), &w = tensor(a[2], 2);
    const Call call(y);
    const int io = io_of(y);
    const int64_t M = y.size(0), N = y.size(1), K = x.size(1), kb = (K + 127) / 128;
    need(is_codes(x) && is_codes(w));
    const void* xp = call.dense(x, x.scalar_type(), {M, K});
    const void* sx = call.dense(a[1], at::kFloat, {M, kb});
    const void* wp = call.dense(w, w.scalar_type(), {N, K});
    const void* sw = call.dense(a[3], at::kFloat, {(N + 127) / 128, kb});
    const void* bias = call.dense_or_none(a[5], at::kFloat, {N});
    void* yp = call.dense(y, y.scalar_type(), {M, N});
    const int32_t dims[3] = {size32(M), size32(N), size32(K)};
    void* stream = call.stream();
    Unlocked unlocked;
    return entries.matmul_fp8(dims, io, xp, static_cast<const float*>(sx), wp,
                              static_cast<const float*>(sw), static_cast<const float*>(bias), yp,
                              stream);
  });
}

// rope(x, freq, pos, q, k, v, interleaved, magnitude, lens)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain([&] {
    need(n == 9);
    const at::Tensor &x = tensor(a[0], 3), &q = tensor(a[3], 4), &k = tensor(a[4], 4);
    const Call call(x);
    const int io = io_of(x);
    const at::ScalarType type = x.scalar_type();
    const int64_t B = x.size(0), T = x.size(1), C = x.size(2);
    const int64_t Hq = q.size(2), D = q.size(3), Hkv = k.size(2);
    need(C == (Hq + (a[5] == Py_None ? 1 : 2) * Hkv) * D);
    int64_t row = C;
    if (!x.is_contiguous()) {
      row = T > 1 ? x.stride(1) : B > 1 ? x.stride(0) : C;
      need((C <= 1 || x.stride(2) == 1) && (T <= 1 || B <= 1 || x.stride(0) == T * row));
    }
    const at::Tensor& f = tensor(a[1], 1);
    const int64_t half = f.size(0);
    const void* freq = call.dense(f, at::kDouble, {half});
    const void* pos = call.dense(a[2], at::kInt, {B});
    const void* lens = call.dense_or_none(a[8], at::kInt, {B});
    void* qp = call.dense(q, type, {B, T, Hq, D});
    void* kp = call.dense(k, type, {B, T, Hkv, D});
    void* vp = call.dense_or_none(a[5], type, {B, T, Hkv, D});
    const int interleaved = PyObject_IsTrue(a[6]);
    const double magnitude = PyFloat_AsDouble(a[7]);
    need(interleaved >= 0 && !PyErr_Occurred());
    const int32_t dims[6] = {size32(B),   size32(T), size32(Hq),
                             size32(Hkv), size32(D), size32(2 * half)};
    const void* xp = x.data_ptr();
    void* stream = call.stream();
    Unlocked unlocked;
    return entries.rope(dims, io, interleaved, xp, row, static_cast<const double*>(freq),
                        static_cast<float>(magnitude), static_cast<const int32_t*>(pos),
                        static_cast<const int32_t*>(lens), qp, kp, vp, stream);
  });
}

PyObject* on_refusal(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(refuse, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ptr)), METH_FASTCALL,
     "Address of a dense tensor of exactly this shape, dtype and device."},
    {"opt", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(opt)), METH_FASTCALL,
     "ptr, or None for None."},
    {"on_refusal", on_refusal, METH_O, "Sets the function that raises for what does not fit."},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL,
     "Takes the library's entry points and torch's accessors."},
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rms_norm)), METH_FASTCALL,
     "gdr_rms_norm's status, or None."},
    {"quant_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_rows)), METH_FASTCALL,
     "gdr_quant_rows's status, or None."},
    {"matmul_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matmul_fp8)), METH_FASTCALL,
     "gdr_matmul_fp8's status, or None."},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL,
     "gdr_rope's status, or None."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
