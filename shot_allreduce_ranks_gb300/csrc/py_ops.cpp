// Python binding of the feed-forward operators (include/ar.h): checks the
// tensors, allocates the outputs that were not given, and calls the C entry
// points on the current stream.
//
// A decoding step's kernels run for a few microseconds, about what a call
// through Python-level checks and ctypes costs the host (11 us a call, of which
// the launch is 2.3); here the checks and allocations are C++, against
// torch's own headers.  feed_forward.py is the public face and documents the
// functions.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "ar.h"

namespace {

PyObject* g_check = nullptr;  // raises ArError for a status and a call's name

struct Refused {
  std::string what;  // becomes a ValueError
};
struct Raised {};  // the Python error is set

[[noreturn]] void refuse(std::string what) { throw Refused{std::move(what)}; }

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kChar: return "torch.int8";
    default: return c10::toString(t);
  }
}

// AR_BF16, AR_FP16 or AR_FP32; half: the first two only.
int type_code(at::ScalarType t, const char* what, bool half) {
  if (t == at::kBFloat16) return AR_BF16;
  if (t == at::kHalf) return AR_FP16;
  if (t == at::kFloat && !half) return AR_FP32;
  refuse(std::string(what) + " must be torch.bfloat16" + (half ? " or torch.float16" : ", torch.float16 or torch.float32") +
         ", got " + type_name(t));
}
at::ScalarType type_of(int code) { return code == AR_BF16 ? at::kBFloat16 : code == AR_FP16 ? at::kHalf : at::kFloat; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", what, Py_TYPE(o)->tp_name);
    throw Raised{};
  }
  return THPVariable_Unpack(o);
}

int gpu_of(const at::Tensor& t, const char* what) {
  if (!t.is_cuda()) refuse(std::string(what) + " must be a CUDA tensor");
  return t.get_device();
}

// A result carries no history, so a gradient that the caller's backward pass
// would have sent to this input is lost: worth a word.
void no_history(const at::Tensor& t, const char* what) {
  if (!t.requires_grad() || !c10::GradMode::is_enabled()) return;
  if (PyErr_WarnFormat(PyExc_UserWarning, 2,
                       "%s requires grad, but torch's differentiation does not record this operator: its result carries "
                       "no gradient. Call the operator's backward pass, and this under torch.no_grad().", what) < 0)
    throw Raised{};
}

constexpr int64_t kAny = -1;

// A matrix on GPU `index`: its leading dimension.
int64_t matrix(const at::Tensor& t, const char* what, at::ScalarType type, int index, int64_t rows = kAny,
               int64_t cols = kAny) {
  if (t.dim() != 2 || t.scalar_type() != type || !t.is_cuda() || t.get_device() != index)
    refuse(std::string(what) + " must be a 2-D " + type_name(type) + " tensor on cuda:" + std::to_string(index));
  const int64_t m = t.size(0), n = t.size(1);
  if ((rows != kAny && m != rows) || (cols != kAny && n != cols))
    refuse(std::string(what) + " must be " + (rows == kAny ? "?" : std::to_string(rows)) + " x " +
           (cols == kAny ? "?" : std::to_string(cols)) + ", got " + std::to_string(m) + " x " + std::to_string(n));
  if (n > 1 && t.stride(1) != 1) refuse(std::string(what) + " must have contiguous rows");
  if (m <= 1) return n;
  if (t.stride(0) < n) refuse(std::string(what) + " has overlapping rows");
  return t.stride(0);
}

void vector(const at::Tensor& t, const char* what, int64_t n, int index) {
  if (t.scalar_type() != at::kFloat || !t.is_cuda() || t.get_device() != index || t.dim() != 1 || t.size(0) != n ||
      !t.is_contiguous())
    refuse(std::string(what) + " must be " + std::to_string(n) + " contiguous float32 values on cuda:" + std::to_string(index));
}

at::Tensor fresh(int64_t rows, int64_t cols, at::ScalarType type, const at::Tensor& like) {
  return at::empty({rows, cols}, like.options().dtype(type));
}

// The given matrix, or a new one; ld receives its leading dimension.
at::Tensor output(PyObject* o, const char* what, at::ScalarType type, int index, int64_t rows, int64_t cols,
                  const at::Tensor& like, int64_t* ld) {
  if (o == Py_None) {
    *ld = cols;
    return fresh(rows, cols, type, like);
  }
  const at::Tensor& t = tensor(o, what);
  *ld = matrix(t, what, type, index, rows, cols);
  return t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
uint64_t unsigned_word(PyObject* o) {
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw Raised{};
    PyErr_Clear();
    refuse("seed, sequence and offset must be in [0, 2^64)");
  }
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
void* handle(PyObject* o) { return reinterpret_cast<void*>(integer(o)); }

// The C call with the tensors' device current, on its current stream.
template <class F>
void call(const char* name, int index, F f) {
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
  void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  ar_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = f(stream);
  Py_END_ALLOW_THREADS;
  if (st != AR_OK) {
    PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, name);
    Py_XDECREF(r);
    throw Raised{};
  }
}

bool unaligned(const at::Tensor& t, int64_t ld, int64_t elem) {
  return ((reinterpret_cast<uintptr_t>(t.data_ptr()) | (uintptr_t)(ld * elem)) & 15) != 0;
}

// Memory in which unaligned rows are laid out; undefined for none.
at::Tensor scratch(size_t bytes, const at::Tensor& like) {
  return bytes ? at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)) : at::Tensor();
}
void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes_of(const at::Tensor& t) { return t.defined() ? (size_t)t.numel() : 0; }

template <class... T>
PyObject* tuple_of(const T&... t) {
  PyObject* items[] = {(t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None))...};
  PyObject* r = PyTuple_New(sizeof...(T));
  for (size_t i = 0; i < sizeof...(T); ++i) {
    if (!r || !items[i]) {
      for (size_t j = i; j < sizeof...(T); ++j) Py_XDECREF(items[j]);
      Py_XDECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i, items[i]);
  }
  return r;
}

// Runs a body that throws the above, and whatever torch throws.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const Raised&) {
  } catch (const c10::Error& e) {
    // Memory that ran out keeps torch's own exception type.
    PyObject* type = nullptr;
    if (dynamic_cast<const c10::OutOfMemoryError*>(&e)) {
      PyObject* torch = PyImport_ImportModule("torch");
      type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
      Py_XDECREF(torch);
      PyErr_Clear();
    }
    PyErr_SetString(type ? type : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(type);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// A GatedFFN's constants: handle, type code, hidden, width, GPU, max_tokens.
struct Ffn {
  ar_ffn_t h;
  at::ScalarType type;
  int64_t hidden, width, max_tokens;
  int index;
  explicit Ffn(PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) {
      PyErr_SetString(PyExc_TypeError, "expected the handle's six constants");
      throw Raised{};
    }
    h = static_cast<ar_ffn_t>(handle(PyTuple_GET_ITEM(o, 0)));
    type = type_of((int)integer(PyTuple_GET_ITEM(o, 1)));
    hidden = integer(PyTuple_GET_ITEM(o, 2));
    width = integer(PyTuple_GET_ITEM(o, 3));
    index = (int)integer(PyTuple_GET_ITEM(o, 4));
    max_tokens = integer(PyTuple_GET_ITEM(o, 5));
  }
};

struct FfnInputs {
  const at::Tensor &x, &wg, &wu;
  int64_t ldx, ldw, m;
  at::Tensor room;
  FfnInputs(const Ffn& f, PyObject* xo, PyObject* wgo, PyObject* wuo, bool backward)
      : x(tensor(xo, "x")), wg(tensor(wgo, "w_gate")), wu(tensor(wuo, "w_up")) {
    ldx = matrix(x, "x", f.type, f.index, kAny, f.hidden);
    ldw = matrix(wg, "w_gate", f.type, f.index, f.width, f.hidden);
    if (matrix(wu, "w_up", f.type, f.index, f.width, f.hidden) != ldw)
      refuse("w_gate and w_up must have the same row stride");
    m = x.size(0);
    if (m <= AR_FEW_TOKENS && !backward) return;  // read as they are
    if (unaligned(x, ldx, 2) || unaligned(wg, ldw, 2) || unaligned(wu, ldw, 2))
      room = scratch(ar_ffn_scratch_bytes(f.h, x.data_ptr(), ldx, wg.data_ptr(), wu.data_ptr(), ldw, m), x);
  }
};

// (constants, x, w_gate, w_up, out, gate, up, save)
PyObject* ffn_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Ffn f(a[0]);
    FfnInputs in(f, a[1], a[2], a[3], false);
    no_history(in.x, "x");
    no_history(in.wg, "w_gate");
    no_history(in.wu, "w_up");
    int64_t ldo;
    const at::Tensor out = output(a[4], "out", f.type, f.index, in.m, f.width, in.x, &ldo);
    at::Tensor gate, up;
    if ((a[5] == Py_None) != (a[6] == Py_None)) refuse("gate and up are given together");
    if (a[5] != Py_None) {
      gate = tensor(a[5], "gate");
      up = tensor(a[6], "up");
      if (matrix(gate, "gate", f.type, f.index, in.m, f.width) != ldo || matrix(up, "up", f.type, f.index, in.m, f.width) != ldo)
        refuse("gate and up must have the row stride of out");
    } else if (PyObject_IsTrue(a[7])) {
      gate = at::empty_strided({in.m, f.width}, {ldo, 1}, in.x.options());
      up = at::empty_strided({in.m, f.width}, {ldo, 1}, in.x.options());
    }
    call("ar_ffn_forward", f.index, [&](void* s) {
      return ar_ffn_forward(f.h, in.x.data_ptr(), in.ldx, in.wg.data_ptr(), in.wu.data_ptr(), in.ldw, out.data_ptr(),
                            address(gate), address(up), ldo, in.m, address(in.room), bytes_of(in.room), s);
    });
    return gate.defined() ? tuple_of(out, gate, up) : THPVariable_Wrap(out);
  });
}

// (constants, x, w_gate, w_up, gate, up, dout, dx, dw_gate, dw_up, need_dx, need_dw)
PyObject* ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Ffn f(a[0]);
    FfnInputs in(f, a[1], a[2], a[3], true);
    if (in.m > f.max_tokens)
      refuse("x has " + std::to_string(in.m) + " rows, the handle's workspace " + std::to_string(f.max_tokens));
    const at::Tensor &gate = tensor(a[4], "gate"), &up = tensor(a[5], "up"), &dout = tensor(a[6], "dout");
    const int64_t ldo = matrix(dout, "dout", f.type, f.index, in.m, f.width);
    if (matrix(gate, "gate", f.type, f.index, in.m, f.width) != ldo || matrix(up, "up", f.type, f.index, in.m, f.width) != ldo)
      refuse("gate, up and dout must have the same row stride");
    at::Tensor dx, dwg, dwu;
    int64_t lddx = f.hidden, lddw = f.hidden, ldu = f.hidden;
    if (PyObject_IsTrue(a[10])) dx = output(a[7], "dx", f.type, f.index, in.m, f.hidden, in.x, &lddx);
    if (PyObject_IsTrue(a[11])) {
      if ((a[8] == Py_None) != (a[9] == Py_None)) refuse("dw_gate and dw_up are given together");
      dwg = output(a[8], "dw_gate", f.type, f.index, f.width, f.hidden, in.x, &lddw);
      dwu = output(a[9], "dw_up", f.type, f.index, f.width, f.hidden, in.x, &ldu);
      if (lddw != ldu) refuse("dw_gate and dw_up must have the same row stride");
    }
    call("ar_ffn_backward", f.index, [&](void* s) {
      return ar_ffn_backward(f.h, in.x.data_ptr(), in.ldx, in.wg.data_ptr(), in.wu.data_ptr(), in.ldw, gate.data_ptr(),
                             up.data_ptr(), dout.data_ptr(), ldo, address(dx), lddx, address(dwg), address(dwu), lddw, in.m,
                             address(in.room), bytes_of(in.room), s);
    });
    return tuple_of(dx, dwg, dwu);
  });
}

// (x, p, seed, sequence, offset, residual, out)
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const int index = gpu_of(x, "x"), code = type_code(x.scalar_type(), "x", false);
    const double p = real(a[1]);
    const uint64_t seed = unsigned_word(a[2]), sequence = unsigned_word(a[3]), offset = unsigned_word(a[4]);
    const int64_t ldx = matrix(x, "x", x.scalar_type(), index), rows = x.size(0), cols = x.size(1);
    no_history(x, "x");
    int64_t ldr = 0, ldo;
    const void* r = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& t = tensor(a[5], "residual");
      ldr = matrix(t, "residual", x.scalar_type(), index, rows, cols);
      no_history(t, "residual");
      r = t.data_ptr();
    }
    const at::Tensor out = output(a[6], "out", x.scalar_type(), index, rows, cols, x, &ldo);
    call("ar_dropout", index, [&](void* s) {
      return ar_dropout(x.data_ptr(), ldx, r, ldr, out.data_ptr(), ldo, rows, cols, code, p, seed, sequence, offset, s);
    });
    return THPVariable_Wrap(out);
  });
}

// (dy, p, seed, sequence, offset, dx)
PyObject* dropout_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor& dy = tensor(a[0], "dy");
    const int index = gpu_of(dy, "dy"), code = type_code(dy.scalar_type(), "dy", false);
    const double p = real(a[1]);
    const uint64_t seed = unsigned_word(a[2]), sequence = unsigned_word(a[3]), offset = unsigned_word(a[4]);
    const int64_t lddy = matrix(dy, "dy", dy.scalar_type(), index), rows = dy.size(0), cols = dy.size(1);
    int64_t lddx;
    const at::Tensor dx = output(a[5], "dx", dy.scalar_type(), index, rows, cols, dy, &lddx);
    call("ar_dropout_backward", index, [&](void* s) {
      return ar_dropout_backward(dy.data_ptr(), lddy, dx.data_ptr(), lddx, rows, cols, code, p, seed, sequence, offset, s);
    });
    return THPVariable_Wrap(dx);
  });
}

// (x, q, scale)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const int index = gpu_of(x, "x"), code = type_code(x.scalar_type(), "x", false);
    const int64_t ldx = matrix(x, "x", x.scalar_type(), index), rows = x.size(0), cols = x.size(1);
    no_history(x, "x");
    int64_t ldq = (cols + 15) / 16 * 16;
    // A new q's rows start on 16 bytes, as the product wants them.
    const at::Tensor q = a[1] != Py_None ? output(a[1], "q", at::kChar, index, rows, cols, x, &ldq)
                         : ldq == cols   ? fresh(rows, cols, at::kChar, x)
                                         : fresh(rows, ldq, at::kChar, x).narrow(1, 0, cols);
    if (rows <= 1 && a[1] == Py_None) ldq = cols;
    at::Tensor scale;
    if (a[2] == Py_None) {
      scale = at::empty({rows}, x.options().dtype(at::kFloat));
    } else {
      scale = tensor(a[2], "scale");
      vector(scale, "scale", rows, index);
    }
    call("ar_quantize_rows", index, [&](void* s) {
      return ar_quantize_rows(x.data_ptr(), ldx, static_cast<int8_t*>(q.data_ptr()), ldq,
                              static_cast<float*>(scale.data_ptr()), rows, cols, code, s);
    });
    return tuple_of(q, scale);
  });
}

// (x, x_scale, w, w_scale, out, type code of a new out)
PyObject* linear_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &sx = tensor(a[1], "x_scale"), &w = tensor(a[2], "w"),
                     &sw = tensor(a[3], "w_scale");
    const int index = gpu_of(x, "x");
    const int64_t ldx = matrix(x, "x", at::kChar, index), rows = x.size(0), in = x.size(1);
    const int64_t ldw = matrix(w, "w", at::kChar, index, kAny, in), cols = w.size(0);
    vector(sx, "x_scale", rows, index);
    vector(sw, "w_scale", cols, index);
    no_history(sx, "x_scale");
    no_history(sw, "w_scale");
    const at::ScalarType type = a[4] == Py_None ? type_of((int)integer(a[5])) : tensor(a[4], "out").scalar_type();
    const int code = type_code(type, "dtype", true);
    int64_t ldy;
    const at::Tensor y = output(a[4], "out", type, index, rows, cols, x, &ldy);
    const int8_t *xp = static_cast<const int8_t*>(x.data_ptr()), *wp = static_cast<const int8_t*>(w.data_ptr());
    at::Tensor room;
    if (unaligned(x, ldx, 1) || unaligned(w, ldw, 1))
      room = scratch(ar_linear_i8_scratch_bytes(xp, ldx, wp, ldw, rows, in, cols), x);
    call("ar_linear_i8", index, [&](void* s) {
      return ar_linear_i8(xp, ldx, static_cast<const float*>(sx.data_ptr()), wp, ldw,
                          static_cast<const float*>(sw.data_ptr()), y.data_ptr(), ldy, rows, in, cols, code, address(room),
                          bytes_of(room), s);
    });
    return THPVariable_Wrap(y);
  });
}

// (check): what raises for a status that is not AR_OK.
PyObject* set_check(PyObject*, PyObject* f) {
  Py_XSETREF(g_check, Py_NewRef(f));
  Py_RETURN_NONE;
}

#define AR_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {AR_FAST(ffn_forward),
                         AR_FAST(ffn_backward),
                         AR_FAST(dropout),
                         AR_FAST(dropout_backward),
                         AR_FAST(quantize_rows),
                         AR_FAST(linear_i8),
                         {"set_check", set_check, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", "Feed-forward operators: see feed_forward.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
