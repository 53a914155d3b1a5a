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
    case at::kByte: return "torch.uint8";
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

void vector(const at::Tensor& t, const char* what, int64_t n, int index, at::ScalarType type = at::kFloat) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != index || t.dim() != 1 || t.size(0) != n ||
      !t.is_contiguous())
    refuse(std::string(what) + " must be " + std::to_string(n) + " contiguous " +
           (type == at::kFloat ? "float32" : type_name(type)) + " values on cuda:" + std::to_string(index));
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

// What a call of the norms has beside its matrices of rows.
struct Norm {
  ar_norm_t n;
  at::ScalarType type;
  int index;
  at::Tensor weight, bias, after_weight, after_bias, gate;
  int64_t ldg = 0;

  // like: a matrix of the call; o: weight, bias, after_weight, after_bias, gate, kind, eps, residual_scale, weight_offset.
  Norm(const at::Tensor& like, const char* what, PyObject* const* o) {
    index = gpu_of(like, what);
    type = like.scalar_type();
    n.dtype = type_code(type, what, false);
    if (like.dim() != 2) refuse(std::string(what) + " must be 2-D");
    n.rows = (size_t)like.size(0), n.cols = (size_t)like.size(1);
    if (n.cols == 0) refuse(std::string(what) + " must have columns");
    weight = one(o[0], "weight"), bias = one(o[1], "bias");
    after_weight = one(o[2], "after_weight"), after_bias = one(o[3], "after_bias");
    if (!weight.defined() && !after_weight.defined()) refuse("weight or after_weight must be given");
    if (bias.defined() && !weight.defined()) refuse("bias needs weight");
    if (after_bias.defined() && !after_weight.defined()) refuse("after_bias needs after_weight");
    n.gate_rows = 0;
    if (o[4] != Py_None) {
      gate = tensor(o[4], "gate");
      ldg = matrix(gate, "gate", type, index, kAny, (int64_t)n.cols);
      n.gate_rows = (size_t)gate.size(0);
      if (n.gate_rows == 0 || n.rows % n.gate_rows)
        refuse("gate has " + std::to_string(n.gate_rows) + " rows, which do not divide " + std::to_string(n.rows));
    }
    n.kind = (int)integer(o[5]);
    n.eps = real(o[6]), n.residual_scale = real(o[7]), n.weight_offset = real(o[8]);
    if (!(n.eps >= 0.0) || n.eps > 3e38) refuse("eps must be finite and not negative");
  }
  at::Tensor one(PyObject* o, const char* what) const {
    if (o == Py_None) return at::Tensor();
    const at::Tensor& t = tensor(o, what);
    vector(t, what, (int64_t)n.cols, index, type);
    return t;
  }
  // A matrix of rows, or null.
  at::Tensor rows(PyObject* o, const char* what, int64_t* ld) const {
    *ld = 0;
    if (o == Py_None) return at::Tensor();
    const at::Tensor& t = tensor(o, what);
    *ld = matrix(t, what, type, index, (int64_t)n.rows, (int64_t)n.cols);
    return t;
  }
};

// (x, residual, weight, bias, after_weight, after_bias, gate, kind, eps, residual_scale, weight_offset, r, y)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 13, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const Norm p(x, "x", a + 2);
    int64_t ldx, ldres, ldr = 0, ldy = 0;
    p.rows(a[0], "x", &ldx);
    const at::Tensor residual = p.rows(a[1], "residual", &ldres);
    no_history(x, "x");
    if (residual.defined()) no_history(residual, "residual");
    if (p.weight.defined()) no_history(p.weight, "weight");
    if (p.bias.defined()) no_history(p.bias, "bias");
    if (p.after_weight.defined()) no_history(p.after_weight, "after_weight");
    if (p.after_bias.defined()) no_history(p.after_bias, "after_bias");
    if (p.gate.defined()) no_history(p.gate, "gate");
    const int64_t m = (int64_t)p.n.rows, n = (int64_t)p.n.cols;
    at::Tensor r, y;
    // Where nothing is added to x and nothing multiplies it, r would be x.
    if (residual.defined() || p.gate.defined() || p.after_weight.defined() || a[11] != Py_None)
      r = output(a[11], "r", p.type, p.index, m, n, x, &ldr);
    if (p.weight.defined())
      y = output(a[12], "y", p.type, p.index, m, n, x, &ldy);
    else if (a[12] != Py_None)
      refuse("y needs weight");
    if (m && r.defined() && y.defined() && r.data_ptr() == y.data_ptr()) refuse("r and y must be two tensors");
    call("ar_residual_norm", p.index, [&](void* s) {
      return ar_residual_norm(&p.n, x.data_ptr(), ldx, address(residual), ldres, address(p.gate), p.ldg, address(p.after_weight),
                              address(p.after_bias), address(p.weight), address(p.bias), address(r), ldr, address(y), ldy, s);
    });
    return tuple_of(r, y);
  });
}

// (dy, dr, x, r, weight, bias, after_weight, after_bias, gate, kind, eps, residual_scale, weight_offset, need_dresidual)
PyObject* residual_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 14, [&]() -> PyObject* {
    const at::Tensor& first = a[0] != Py_None ? tensor(a[0], "dy") : tensor(a[1], "dr");
    const Norm p(first, a[0] != Py_None ? "dy" : "dr", a + 4);
    const int64_t m = (int64_t)p.n.rows, n = (int64_t)p.n.cols;
    int64_t lddy, lddr, ldx, ldr;
    const at::Tensor dy = p.rows(a[0], "dy", &lddy), dr = p.rows(a[1], "dr", &lddr), x = p.rows(a[2], "x", &ldx);
    at::Tensor r = p.rows(a[3], "r", &ldr);
    const bool branch = p.gate.defined() || p.after_weight.defined();
    if (dy.defined() != p.weight.defined()) refuse("dy and weight are given together");
    if (branch && !x.defined()) refuse("a gate or after_weight needs x");
    const bool added = r.defined();
    if (p.weight.defined() && !added) {
      if (branch || !x.defined()) refuse("weight needs r");
      r = x, ldr = ldx;  // nothing was added
    }
    const at::Tensor& like = first;
    const at::Tensor dx = fresh(m, n, p.type, like);
    at::Tensor dres;
    // The gradient of the residual is that of x where nothing stands between them.
    const bool same = !branch && p.n.residual_scale == 1.0;
    const bool need = added && PyObject_IsTrue(a[13]);
    if (need && !same) dres = fresh(m, n, p.type, like);
    const auto param = [&](const at::Tensor& t) { return t.defined() ? at::empty({n}, like.options()) : at::Tensor(); };
    const at::Tensor dw = param(p.weight), db = param(p.bias), daw = param(p.after_weight), dab = param(p.after_bias);
    const at::Tensor dgate = p.gate.defined() ? fresh((int64_t)p.n.gate_rows, n, p.type, like) : at::Tensor();
    const int vectors = dw.defined() + db.defined() + daw.defined() + dab.defined() + dgate.defined();
    const at::Tensor room = scratch(ar_residual_norm_scratch_bytes(p.n.rows, p.n.cols, vectors), like);
    call("ar_residual_norm_backward", p.index, [&](void* s) {
      return ar_residual_norm_backward(&p.n, address(dy), lddy, address(dr), lddr, address(x), ldx, address(r), ldr,
                                       address(p.gate), p.ldg, address(p.after_weight), address(p.after_bias), address(p.weight),
                                       address(dx), n, address(dres), n, address(dgate), n, address(dw), address(db), address(daw),
                                       address(dab), address(room), bytes_of(room), s);
    });
    return tuple_of(dx, need && same ? dx : dres, dw, db, daw, dab, dgate);
  });
}

// An Int4Weight's constants: data, scale, zero or None, out, in, group.
struct Packed {
  at::Tensor data, scale, zero;
  int64_t out, in;
  int group, index, code;
  at::ScalarType type;
  explicit Packed(PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) {
      PyErr_SetString(PyExc_TypeError, "expected an Int4Weight's six constants");
      throw Raised{};
    }
    data = tensor(PyTuple_GET_ITEM(o, 0), "data"), scale = tensor(PyTuple_GET_ITEM(o, 1), "scale");
    if (PyTuple_GET_ITEM(o, 2) != Py_None) zero = tensor(PyTuple_GET_ITEM(o, 2), "zero");
    out = integer(PyTuple_GET_ITEM(o, 3)), in = integer(PyTuple_GET_ITEM(o, 4)), group = (int)integer(PyTuple_GET_ITEM(o, 5));
    index = gpu_of(data, "data"), type = scale.scalar_type(), code = type_code(type, "scale", true);
    size_t bytes = 0, scales = 0;
    if (ar_i4_sizes((size_t)out, (size_t)in, group, &bytes, &scales) != AR_OK) refuse("an Int4Weight of no matrix's size");
    array(data, "data", at::kByte, bytes);
    array(scale, "scale", type, scales);
    if (zero.defined()) array(zero, "zero", at::kByte, scales);
  }
  void array(const at::Tensor& t, const char* what, at::ScalarType want, size_t count) const {
    if (t.scalar_type() != want || !t.is_cuda() || t.get_device() != index || !t.is_contiguous() || (size_t)t.numel() != count)
      refuse(std::string("the weight's ") + what + " must be " + std::to_string(count) + " contiguous " + type_name(want) +
             " values on cuda:" + std::to_string(index));
  }
  // New arrays for a layout.
  Packed(int64_t out_, int64_t in_, int group_, bool zeros, at::ScalarType type_, const at::Tensor& like)
      : out(out_), in(in_), group(group_), index(like.get_device()), type(type_) {
    if (group != 32 && group != 64 && group != 128) refuse("group must be 32, 64 or 128");
    size_t bytes = 0, scales = 0;
    if (ar_i4_sizes((size_t)out, (size_t)in, group, &bytes, &scales) != AR_OK)
      refuse("weights must have 1 to 2^30 rows and columns, got " + std::to_string(out) + " x " + std::to_string(in));
    code = type_code(type, "scale", true);
    data = at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
    scale = at::empty({(int64_t)scales}, like.options().dtype(type));
    if (zeros) zero = at::empty({(int64_t)scales}, like.options().dtype(at::kByte));
  }
};

// (q, scale, zero, group): data, scale, zero
PyObject* pack_i4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &scale = tensor(a[1], "scale");
    const int index = gpu_of(q, "q"), group = (int)integer(a[3]);
    if (group != 32 && group != 64 && group != 128) refuse("group must be 32, 64 or 128");
    const int64_t ldq = matrix(q, "q", at::kByte, index), rows = q.size(0), cols = q.size(1), groups = (cols + group - 1) / group;
    const at::ScalarType type = scale.scalar_type();
    type_code(type, "scale", true);
    const int64_t lds = matrix(scale, "scale", type, index, rows, groups);
    int64_t ldz = 0;
    at::Tensor zero;
    if (a[2] != Py_None) {
      zero = tensor(a[2], "zero");
      ldz = matrix(zero, "zero", at::kByte, index, rows, groups);
    }
    no_history(scale, "scale");
    const Packed p(rows, cols, group, zero.defined(), type, q);
    call("ar_pack_i4", index, [&](void* s) {
      return ar_pack_i4(static_cast<const uint8_t*>(q.data_ptr()), ldq, scale.data_ptr(), lds, static_cast<const uint8_t*>(address(zero)),
                        ldz, rows, cols, group, p.data.data_ptr(), p.scale.data_ptr(), address(p.zero), s);
    });
    return tuple_of(p.data, p.scale, p.zero);
  });
}

// (w, group, whether zero points): data, scale, zero
PyObject* quantize_i4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    const at::Tensor& w = tensor(a[0], "w");
    const int index = gpu_of(w, "w");
    const at::ScalarType type = w.scalar_type();
    const int code = type_code(type, "w", true);
    const int64_t ldw = matrix(w, "w", type, index), rows = w.size(0), cols = w.size(1);
    no_history(w, "w");
    const Packed p(rows, cols, (int)integer(a[1]), PyObject_IsTrue(a[2]), type, w);
    const at::Tensor room = scratch(ar_quantize_i4_scratch_bytes(rows, cols, p.group), w);
    call("ar_quantize_i4", index, [&](void* s) {
      return ar_quantize_i4(w.data_ptr(), ldw, rows, cols, p.group, code, p.data.data_ptr(), p.scale.data_ptr(), address(p.zero),
                            address(room), bytes_of(room), s);
    });
    return tuple_of(p.data, p.scale, p.zero);
  });
}

// (constants, out)
PyObject* dequantize_i4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    const Packed p(a[0]);
    int64_t ldw;
    const at::Tensor w = output(a[1], "out", p.type, p.index, p.out, p.in, p.scale, &ldw);
    call("ar_dequantize_i4", p.index, [&](void* s) {
      return ar_dequantize_i4(p.data.data_ptr(), p.scale.data_ptr(), address(p.zero), p.out, p.in, p.group, p.code, w.data_ptr(), ldw, s);
    });
    return THPVariable_Wrap(w);
  });
}

// (x, constants, out)
PyObject* linear_i4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    const Packed p(a[1]);
    const at::Tensor& x = tensor(a[0], "x");
    const int64_t ldx = matrix(x, "x", p.type, p.index, kAny, p.in), rows = x.size(0);
    no_history(x, "x");
    int64_t ldy;
    const at::Tensor y = output(a[2], "out", p.type, p.index, rows, p.out, x, &ldy);
    call("ar_linear_i4", p.index, [&](void* s) {
      return ar_linear_i4(x.data_ptr(), ldx, p.data.data_ptr(), p.scale.data_ptr(), address(p.zero), y.data_ptr(), ldy, rows, p.in,
                          p.out, p.group, p.code, s);
    });
    return THPVariable_Wrap(y);
  });
}

// Experts' matrices: row and expert strides.
const at::Tensor& stack(PyObject* o, const char* what, at::ScalarType type, int index, int64_t count, int64_t rows, int64_t cols,
                        int64_t* ld, int64_t* es) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 3 || t.scalar_type() != type || !t.is_cuda() || t.get_device() != index)
    refuse(std::string(what) + " must be a 3-D " + type_name(type) + " tensor on cuda:" + std::to_string(index));
  const int64_t want[3] = {count, rows, cols};
  for (int i = 0; i < 3; ++i)
    if (want[i] != kAny && t.size(i) != want[i])
      refuse(std::string(what) + " has size " + std::to_string(t.size(i)) + " in dimension " + std::to_string(i) + ", wanted " +
             std::to_string(want[i]));
  if (t.numel() == 0) refuse(std::string(what) + " is empty");
  if (t.size(2) > 1 && t.stride(2) != 1) refuse(std::string(what) + " must have contiguous rows");
  *ld = t.size(1) > 1 ? t.stride(1) : t.size(2);
  if (*ld < t.size(2)) refuse(std::string(what) + " has overlapping rows");
  *es = t.size(0) > 1 ? t.stride(0) : 0;
  return t;
}

// (x, logits, w_gate, w_up, w_down, top_k, activation, normalize, first_expert, out, routing)
PyObject* moe_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &logits = tensor(a[1], "logits");
    const int index = gpu_of(x, "x");
    ar_moe_t m = {};
    m.dtype = type_code(x.scalar_type(), "x", true);
    m.logits_dtype = type_code(logits.scalar_type(), "logits", false);
    const int64_t ldx = matrix(x, "x", x.scalar_type(), index), rows = x.size(0), K = x.size(1);
    const int64_t ldl = matrix(logits, "logits", logits.scalar_type(), index, rows);
    int64_t ldw, esw, ldu, esu, ldd, esd, ldo;
    const at::Tensor& wg = stack(a[2], "w_gate", x.scalar_type(), index, kAny, kAny, K, &ldw, &esw);
    const int64_t local = wg.size(0), F = wg.size(1);
    const at::Tensor& wu = stack(a[3], "w_up", x.scalar_type(), index, local, F, K, &ldu, &esu);
    if (ldu != ldw || esu != esw) refuse("w_gate and w_up must have the same strides");
    const at::Tensor& wd = stack(a[4], "w_down", x.scalar_type(), index, local, K, F, &ldd, &esd);
    for (int i = 0; i < 5; ++i) {
      static const char* const names[] = {"x", "logits", "w_gate", "w_up", "w_down"};
      no_history(tensor(a[i], names[i]), names[i]);
    }
    const int64_t experts = logits.size(1), top_k = integer(a[5]), first = integer(a[8]);
    if (experts < 1 || experts > AR_MAX_EXPERTS) refuse("logits must have 1 to " + std::to_string(AR_MAX_EXPERTS) + " columns");
    if (first < 0 || first > experts - local)
      refuse("experts " + std::to_string(first) + " to " + std::to_string(first + local - 1) + " are not among the " +
             std::to_string(experts) + " of the logits");
    if (top_k < 1 || top_k > experts || top_k > AR_MAX_TOP_K)
      refuse("top_k must be in 1 to " + std::to_string(experts < AR_MAX_TOP_K ? experts : (int64_t)AR_MAX_TOP_K));
    m.activation = (int)integer(a[6]), m.normalize = PyObject_IsTrue(a[7]);
    m.experts = (int)experts, m.first_expert = (int)first, m.local_experts = (int)local, m.top_k = (int)top_k;
    m.hidden = (size_t)K, m.width = (size_t)F;
    const at::Tensor out = output(a[9], "out", x.scalar_type(), index, rows, K, x, &ldo);
    at::Tensor expert, weight;
    if (PyObject_IsTrue(a[10])) {
      expert = at::empty({rows, top_k}, x.options().dtype(at::kInt));
      weight = at::empty({rows, top_k}, x.options().dtype(at::kFloat));
    }
    const at::Tensor room = scratch(ar_moe_two_part_scratch_bytes(&m, (size_t)rows), x);
    call("ar_moe_ffn", index, [&](void* s) {
      return ar_moe_ffn(&m, x.data_ptr(), ldx, logits.data_ptr(), ldl, wg.data_ptr(), wu.data_ptr(), ldw, esw, wd.data_ptr(), ldd,
                        esd, out.data_ptr(), ldo, static_cast<int32_t*>(address(expert)), static_cast<float*>(address(weight)),
                        (size_t)rows, address(room), bytes_of(room), s);
    });
    return expert.defined() ? tuple_of(out, expert, weight) : THPVariable_Wrap(out);
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
                         AR_FAST(pack_i4),
                         AR_FAST(quantize_i4),
                         AR_FAST(dequantize_i4),
                         AR_FAST(linear_i4),
                         AR_FAST(moe_ffn),
                         AR_FAST(residual_norm),
                         AR_FAST(residual_norm_backward),
                         {"set_check", set_check, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", "Feed-forward operators: see feed_forward.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
