"""Feed-forward operators around the sum over ranks (contracts in include/ar.h).

``GatedFFN`` is one rank's shard of the gated projections with its gradients,
``linear_i8`` (with ``quantize_rows``) the down projection in 8-bit integers,
``dropout`` the step after the sum, its mask drawn from the elements' places
and never stored.  Matrices are 2-D CUDA tensors whose rows are contiguous
(any row stride).  Calls are asynchronous on the current (or given) stream,
which also owns the outputs that a call allocates, and run on the tensors'
device.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import ACTIVATIONS, AR_BF16, AR_FP16, AR_FP32, check, load

_CODES = {torch.bfloat16: AR_BF16, torch.float16: AR_FP16, torch.float32: AR_FP32}
_U64 = (1 << 64) - 1

# A call costs the host a few microseconds, which is what a single token's
# step costs the GPU, so the checks below are kept short.
_get_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_functions = None


def _lib():
    global _functions
    if _functions is None:
        _functions = load()
    return _functions


def _code(dtype, what: str, half: bool = False) -> int:
    code = _CODES.get(dtype)
    if code is None or (half and code == AR_FP32):
        raise ValueError("%s must be torch.bfloat16%s, got %s"
                         % (what, " or torch.float16" if half else ", torch.float16 or torch.float32", dtype))
    return code


def _matrix(t, what: str, dtype, index: int, rows=None, cols=None) -> int:
    """Checks a matrix on GPU `index` and gives its leading dimension."""
    shape = t.shape
    if t.dtype is not dtype or t.get_device() != index or len(shape) != 2:
        raise ValueError("%s must be a 2-D %s tensor on cuda:%d" % (what, dtype, index))
    m, n = shape
    if (rows is not None and m != rows) or (cols is not None and n != cols):
        raise ValueError("%s must be %s x %s, got %d x %d"
                         % (what, "?" if rows is None else rows, "?" if cols is None else cols, m, n))
    step, inner = t.stride()
    if inner != 1 and n > 1:
        raise ValueError("%s must have contiguous rows" % what)
    if m <= 1:
        return n
    if step < n:
        raise ValueError("%s has overlapping rows" % what)
    return step


def _on_gpu(t, what: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError("%s must be a CUDA tensor" % what)
    return index


def _call(name: str, index: int, *args) -> None:
    """The C call on the current stream, with the tensors' device current."""
    fn = getattr(_functions or _lib(), name)
    s = _raw_stream(index)
    if index == _get_device():
        status = fn(*args, s)
    else:
        with torch.cuda.device(index):
            status = fn(*args, s)
    if status:
        check(status, name)


def _scratch(name: str, device, *args):
    """(address, bytes, tensor) of the memory in which unaligned rows are laid out."""
    n = getattr(_functions or _lib(), name)(*args)
    t = torch.empty(n, dtype=torch.uint8, device=device)
    return t.data_ptr(), n, t


class GatedFFN:
    """One rank's gated feed-forward shard: ``act(x Wgate^T) * (x Wup^T)``.

    ``hidden`` is the width of x, ``width`` this rank's rows of both weight
    matrices.  ``train=True`` also allocates the workspace of ``backward`` for
    up to ``max_tokens`` rows; without it ``backward`` is refused.
    ``backward`` calls share that workspace: order them on one stream.
    """

    def __init__(self, max_tokens: int, hidden: int, width: int, dtype=torch.bfloat16,
                 activation: str = "silu", train: bool = False, device=None):
        lib = load()
        if activation not in ACTIVATIONS:
            raise ValueError("activation must be one of %s" % ", ".join(sorted(ACTIVATIONS)))
        self.max_tokens, self.hidden, self.width = int(max_tokens), int(hidden), int(width)
        self.dtype, self.train = dtype, bool(train)
        if min(self.max_tokens, self.hidden, self.width) < 1:
            raise ValueError("max_tokens, hidden and width must be at least 1")
        code = _code(dtype, "dtype", half=True)
        index = None if device is None else torch.device(device).index
        self.device = torch.device("cuda", torch.cuda.current_device() if index is None else index)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib.ar_ffn_create(self.max_tokens, self.hidden, self.width, code,
                                          ACTIVATIONS[activation], int(self.train),
                                          ctypes.byref(h)), "ar_ffn_create")
        self._h = h
        self._index = self.device.index

    def close(self) -> None:
        if getattr(self, "_h", None):
            with torch.cuda.device(self.device):
                check(load().ar_ffn_destroy(self._h), "ar_ffn_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _weights(self, w_gate, w_up) -> int:
        ld = _matrix(w_gate, "w_gate", self.dtype, self._index, self.width, self.hidden)
        if _matrix(w_up, "w_up", self.dtype, self._index, self.width, self.hidden) != ld:
            raise ValueError("w_gate and w_up must have the same row stride")
        return ld

    def forward(self, x, w_gate, w_up, out=None, gate=None, up=None, save: bool = False, stream=None):
        """``out``; with ``save`` (or given ``gate`` and ``up``) ``(out, gate, up)``."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, w_gate, w_up, out, gate, up, save)
        dt, index, width = self.dtype, self._index, self.width
        ldx = _matrix(x, "x", dt, index, None, self.hidden)
        ldw = self._weights(w_gate, w_up)
        m = x.shape[0]
        if out is None:
            out, ldo = torch.empty((m, width), dtype=dt, device=self.device), width
        else:
            ldo = _matrix(out, "out", dt, index, m, width)
        g = u = None
        if save or gate is not None or up is not None:
            if (gate is None) != (up is None):
                raise ValueError("gate and up are given together")
            save = True
            if gate is None:
                gate, up = (torch.empty_strided((m, width), (ldo, 1), dtype=dt, device=self.device) for _ in "gu")
            elif _matrix(gate, "gate", dt, index, m, width) != ldo or _matrix(up, "up", dt, index, m, width) != ldo:
                raise ValueError("gate and up must have the row stride of out")
            g, u = gate.data_ptr(), up.data_ptr()
        xp, wg, wu = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
        scratch = None, 0
        if (xp | wg | wu | ldx * 2 | ldw * 2) & 15:
            scratch = _scratch("ar_ffn_scratch_bytes", x.device, self._h, xp, ldx, wg, wu, ldw, m)
        _call("ar_ffn_forward", index, self._h, xp, ldx, wg, wu, ldw, out.data_ptr(), g, u, ldo, m, scratch[0],
              scratch[1])
        return (out, gate, up) if save else out

    def backward(self, x, w_gate, w_up, gate, up, dout, dx=None, dw_gate=None, dw_up=None,
                 need_dx: bool = True, need_dw: bool = True, stream=None):
        """``(dx, dw_gate, dw_up)`` from the saved ``gate`` and ``up``; None for what is not needed."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(x, w_gate, w_up, gate, up, dout, dx, dw_gate, dw_up, need_dx, need_dw)
        dt, index, hidden, width = self.dtype, self._index, self.hidden, self.width
        ldx = _matrix(x, "x", dt, index, None, hidden)
        ldw = self._weights(w_gate, w_up)
        m = x.shape[0]
        if m > self.max_tokens:
            raise ValueError("x has %d rows, the handle's workspace %d" % (m, self.max_tokens))
        ldo = _matrix(dout, "dout", dt, index, m, width)
        if _matrix(gate, "gate", dt, index, m, width) != ldo or _matrix(up, "up", dt, index, m, width) != ldo:
            raise ValueError("gate, up and dout must have the same row stride")
        lddx = lddw = hidden
        if not need_dx:
            dx = None
        elif dx is None:
            dx = torch.empty((m, hidden), dtype=dt, device=self.device)
        else:
            lddx = _matrix(dx, "dx", dt, index, m, hidden)
        if not need_dw:
            dw_gate = dw_up = None
        elif dw_gate is None and dw_up is None:
            dw_gate, dw_up = (torch.empty((width, hidden), dtype=dt, device=self.device) for _ in "gu")
        else:
            if dw_gate is None or dw_up is None:
                raise ValueError("dw_gate and dw_up are given together")
            lddw = _matrix(dw_gate, "dw_gate", dt, index, width, hidden)
            if _matrix(dw_up, "dw_up", dt, index, width, hidden) != lddw:
                raise ValueError("dw_gate and dw_up must have the same row stride")
        xp, wg, wu = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
        scratch = None, 0
        if (xp | wg | wu | ldx * 2 | ldw * 2) & 15:
            scratch = _scratch("ar_ffn_scratch_bytes", x.device, self._h, xp, ldx, wg, wu, ldw, m)
        _call("ar_ffn_backward", index, self._h, xp, ldx, wg, wu, ldw,
              gate.data_ptr(), up.data_ptr(), dout.data_ptr(), ldo, dx.data_ptr() if need_dx else None, lddx,
              dw_gate.data_ptr() if need_dw else None, dw_up.data_ptr() if need_dw else None, lddw, m, scratch[0],
              scratch[1])
        return dx, dw_gate, dw_up


def _draw_args(seed, sequence, offset) -> None:
    if not (0 <= seed <= _U64 and 0 <= sequence <= _U64 and 0 <= offset <= _U64):
        raise ValueError("seed, sequence and offset must be in [0, 2^64)")


def dropout(x, p: float, seed: int, sequence: int = 0, offset: int = 0, residual=None, out=None,
            stream=None):
    """``residual + (keep ? x / (1 - p) : 0)``, the mask drawn from each element's place.

    Element (i, j) draws at ``offset + i * cols + j`` of the stream that
    ``seed`` and ``sequence`` name; equal arguments draw equal masks.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return dropout(x, p, seed, sequence, offset, residual, out)
    index, dt = _on_gpu(x, "x"), x.dtype
    code = _code(dt, "x")
    _draw_args(seed, sequence, offset)
    ldx = _matrix(x, "x", dt, index)
    m, n = x.shape
    r, ldr = None, 0
    if residual is not None:
        r, ldr = residual.data_ptr(), _matrix(residual, "residual", dt, index, m, n)
    if out is None:
        out, ldo = torch.empty((m, n), dtype=dt, device=x.device), n
    else:
        ldo = _matrix(out, "out", dt, index, m, n)
    _call("ar_dropout", index, x.data_ptr(), ldx, r, ldr, out.data_ptr(), ldo, m, n, code, p, seed,
          sequence, offset)
    return out


def dropout_backward(dy, p: float, seed: int, sequence: int = 0, offset: int = 0, dx=None, stream=None):
    """Gradient of ``dropout`` with respect to x (that of ``residual`` is dy)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dropout_backward(dy, p, seed, sequence, offset, dx)
    index, dt = _on_gpu(dy, "dy"), dy.dtype
    code = _code(dt, "dy")
    _draw_args(seed, sequence, offset)
    lddy = _matrix(dy, "dy", dt, index)
    m, n = dy.shape
    if dx is None:
        dx, lddx = torch.empty((m, n), dtype=dt, device=dy.device), n
    else:
        lddx = _matrix(dx, "dx", dt, index, m, n)
    _call("ar_dropout_backward", index, dy.data_ptr(), lddy, dx.data_ptr(), lddx, m, n, code, p, seed,
          sequence, offset)
    return dx


def _vector(t, what: str, n: int, index: int) -> None:
    if t.dtype is not torch.float32 or t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be %d contiguous float32 values on cuda:%d" % (what, n, index))


def quantize_rows(x, q=None, scale=None, stream=None):
    """``(q, scale)``: ``scale[i] = max |x[i]| / 127``, ``q = rint(x / scale)`` in int8."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_rows(x, q, scale)
    index, dt = _on_gpu(x, "x"), x.dtype
    code = _code(dt, "x")
    ldx = _matrix(x, "x", dt, index)
    m, n = x.shape
    if q is None:
        q, ldq = torch.empty((m, n), dtype=torch.int8, device=x.device), n
    else:
        ldq = _matrix(q, "q", torch.int8, index, m, n)
    if scale is None:
        scale = torch.empty(m, dtype=torch.float32, device=x.device)
    else:
        _vector(scale, "scale", m, index)
    _call("ar_quantize_rows", index, x.data_ptr(), ldx, q.data_ptr(), ldq, scale.data_ptr(), m, n, code)
    return q, scale


def linear_i8(x, x_scale, w, w_scale, out=None, dtype=torch.bfloat16, stream=None):
    """``x_scale[m] * w_scale[n] * sum_k x[m, k] w[n, k]`` of int8 matrices, rounded to ``dtype``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_i8(x, x_scale, w, w_scale, out, dtype)
    index = _on_gpu(x, "x")
    ldx = _matrix(x, "x", torch.int8, index)
    m, k = x.shape
    ldw = _matrix(w, "w", torch.int8, index, None, k)
    n = w.shape[0]
    _vector(x_scale, "x_scale", m, index)
    _vector(w_scale, "w_scale", n, index)
    code = _code(dtype if out is None else out.dtype, "dtype", half=True)
    if out is None:
        out, ldo = torch.empty((m, n), dtype=dtype, device=x.device), n
    else:
        ldo = _matrix(out, "out", out.dtype, index, m, n)
    xp, wp, scratch = x.data_ptr(), w.data_ptr(), (None, 0)
    if (xp | wp | ldx | ldw) & 15:
        scratch = _scratch("ar_linear_i8_scratch_bytes", x.device, xp, ldx, wp, ldw, m, k, n)
    _call("ar_linear_i8", index, xp, ldx, x_scale.data_ptr(), wp, ldw, w_scale.data_ptr(), out.data_ptr(), ldo, m, k,
          n, code, scratch[0], scratch[1])
    return out


def ops_device_status(stream=None) -> int:
    """AR_OK, or AR_ERR_TIMEOUT if a wait in one of these operators' kernels gave up (clears it)."""
    s = torch.cuda.current_stream() if stream is None else stream
    return _lib().ar_ops_get_device_status(s.cuda_stream)
