"""Feed-forward operators around the sum over ranks (contracts in include/ar.h).

``GatedFFN`` is one rank's shard of the gated projections with its gradients,
``linear_i8`` (with ``quantize_rows``) the down projection in 8-bit integers,
``dropout`` the step after the sum, its mask drawn from the elements' places
and never stored.  Matrices are 2-D CUDA tensors whose rows are contiguous
(any row stride).  Calls are asynchronous on the current (or given) stream and
run on the tensors' device.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import ACTIVATIONS, AR_BF16, AR_FP16, AR_FP32, check, load

_CODES = {torch.bfloat16: AR_BF16, torch.float16: AR_FP16, torch.float32: AR_FP32}
_U64 = (1 << 64) - 1


def _code(dtype, what: str, half: bool = False) -> int:
    code = _CODES.get(dtype)
    if code is None or (half and code == AR_FP32):
        raise ValueError("%s must be torch.bfloat16%s, got %s"
                         % (what, " or torch.float16" if half else ", torch.float16 or torch.float32", dtype))
    return code


def _matrix(t, what: str, dtype, device, rows=None, cols=None) -> int:
    """Checks a matrix and gives its leading dimension."""
    if t.dim() != 2 or t.dtype != dtype or t.device != device:
        raise ValueError("%s must be a 2-D %s tensor on %s" % (what, dtype, device))
    m, n = t.shape
    if (rows is not None and m != rows) or (cols is not None and n != cols):
        raise ValueError("%s must be %s x %s, got %d x %d"
                         % (what, "?" if rows is None else rows, "?" if cols is None else cols, m, n))
    step, inner = t.stride()
    if n > 1 and inner != 1:
        raise ValueError("%s must have contiguous rows" % what)
    if m <= 1:
        return n
    if step < n:
        raise ValueError("%s has overlapping rows" % what)
    return step


def _on_gpu(t, what: str):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    return t.device


def _launch(device, stream, call, what: str) -> None:
    """call(stream handle) with the tensors' device current."""
    if device.index == torch.cuda.current_device():
        s = torch.cuda.current_stream() if stream is None else stream
        check(call(s.cuda_stream), what)
        return
    with torch.cuda.device(device):
        s = torch.cuda.current_stream() if stream is None else stream
        check(call(s.cuda_stream), what)


class GatedFFN:
    """One rank's gated feed-forward shard: ``act(x Wgate^T) * (x Wup^T)``.

    ``hidden`` is the width of x, ``width`` this rank's rows of both weight
    matrices.  ``train=True`` also allocates the workspace of ``backward`` for
    up to ``max_tokens`` rows; without it ``backward`` is refused.
    ``backward`` calls share that workspace: order them on one stream.
    """

    def __init__(self, max_tokens: int, hidden: int, width: int, dtype=torch.bfloat16,
                 activation: str = "silu", train: bool = False, device=None):
        self._lib = load()
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
            check(self._lib.ar_ffn_create(self.max_tokens, self.hidden, self.width, code,
                                          ACTIVATIONS[activation], int(self.train),
                                          ctypes.byref(h)), "ar_ffn_create")
        self._h = h

    def close(self) -> None:
        if getattr(self, "_h", None):
            with torch.cuda.device(self.device):
                check(self._lib.ar_ffn_destroy(self._h), "ar_ffn_destroy")
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
        ld = _matrix(w_gate, "w_gate", self.dtype, self.device, self.width, self.hidden)
        if _matrix(w_up, "w_up", self.dtype, self.device, self.width, self.hidden) != ld:
            raise ValueError("w_gate and w_up must have the same row stride")
        return ld

    def forward(self, x, w_gate, w_up, out=None, gate=None, up=None, save: bool = False, stream=None):
        """``out``; with ``save`` (or given ``gate`` and ``up``) ``(out, gate, up)``."""
        ldx = _matrix(x, "x", self.dtype, self.device, None, self.hidden)
        ldw = self._weights(w_gate, w_up)
        m = x.shape[0]
        if (gate is None) != (up is None):
            raise ValueError("gate and up are given together")
        save = save or gate is not None
        if out is None:
            out = torch.empty((m, self.width), dtype=self.dtype, device=self.device)
        ldo = _matrix(out, "out", self.dtype, self.device, m, self.width)
        if save:
            if gate is None:
                gate = torch.empty_strided(out.shape, out.stride(), dtype=self.dtype, device=self.device)
                up = torch.empty_strided(out.shape, out.stride(), dtype=self.dtype, device=self.device)
            for t, what in ((gate, "gate"), (up, "up")):
                if _matrix(t, what, self.dtype, self.device, m, self.width) != ldo:
                    raise ValueError("%s must have the row stride of out" % what)
        _launch(self.device, stream, lambda s: self._lib.ar_ffn_forward(
            self._h, x.data_ptr(), ldx, w_gate.data_ptr(), w_up.data_ptr(), ldw, out.data_ptr(),
            gate.data_ptr() if save else None, up.data_ptr() if save else None, ldo, m, s),
            "ar_ffn_forward")
        return (out, gate, up) if save else out

    def backward(self, x, w_gate, w_up, gate, up, dout, dx=None, dw_gate=None, dw_up=None,
                 need_dx: bool = True, need_dw: bool = True, stream=None):
        """``(dx, dw_gate, dw_up)`` from the saved ``gate`` and ``up``; None for what is not needed."""
        dev, dt = self.device, self.dtype
        ldx = _matrix(x, "x", dt, dev, None, self.hidden)
        ldw = self._weights(w_gate, w_up)
        m = x.shape[0]
        if m > self.max_tokens:
            raise ValueError("x has %d rows, the handle's workspace %d" % (m, self.max_tokens))
        ldo = _matrix(dout, "dout", dt, dev, m, self.width)
        if (_matrix(gate, "gate", dt, dev, m, self.width) != ldo
                or _matrix(up, "up", dt, dev, m, self.width) != ldo):
            raise ValueError("gate, up and dout must have the same row stride")
        lddx = lddw = 0
        if need_dx:
            dx = torch.empty((m, self.hidden), dtype=dt, device=dev) if dx is None else dx
            lddx = _matrix(dx, "dx", dt, dev, m, self.hidden)
        if need_dw:
            if (dw_gate is None) != (dw_up is None):
                raise ValueError("dw_gate and dw_up are given together")
            if dw_gate is None:
                dw_gate = torch.empty((self.width, self.hidden), dtype=dt, device=dev)
                dw_up = torch.empty((self.width, self.hidden), dtype=dt, device=dev)
            lddw = _matrix(dw_gate, "dw_gate", dt, dev, self.width, self.hidden)
            if _matrix(dw_up, "dw_up", dt, dev, self.width, self.hidden) != lddw:
                raise ValueError("dw_gate and dw_up must have the same row stride")
        _launch(dev, stream, lambda s: self._lib.ar_ffn_backward(
            self._h, x.data_ptr(), ldx, w_gate.data_ptr(), w_up.data_ptr(), ldw, gate.data_ptr(),
            up.data_ptr(), dout.data_ptr(), ldo, dx.data_ptr() if need_dx else None, lddx,
            dw_gate.data_ptr() if need_dw else None, dw_up.data_ptr() if need_dw else None, lddw,
            m, s), "ar_ffn_backward")
        return dx if need_dx else None, dw_gate if need_dw else None, dw_up if need_dw else None


def _dropout_args(x, seed, sequence, offset):
    _on_gpu(x, "x")
    code = _code(x.dtype, "x")
    for v, what in ((seed, "seed"), (sequence, "sequence"), (offset, "offset")):
        if not 0 <= v <= _U64:
            raise ValueError("%s must be in [0, 2^64)" % what)
    return code


def dropout(x, p: float, seed: int, sequence: int = 0, offset: int = 0, residual=None, out=None,
            stream=None):
    """``residual + (keep ? x / (1 - p) : 0)``, the mask drawn from each element's place.

    Element (i, j) draws at ``offset + i * cols + j`` of the stream that
    ``seed`` and ``sequence`` name; equal arguments draw equal masks.
    """
    code = _dropout_args(x, seed, sequence, offset)
    ldx = _matrix(x, "x", x.dtype, x.device)
    m, n = x.shape
    ldr = 0 if residual is None else _matrix(residual, "residual", x.dtype, x.device, m, n)
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    ldo = _matrix(out, "out", x.dtype, x.device, m, n)
    lib = load()
    _launch(x.device, stream, lambda s: lib.ar_dropout(
        x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, out.data_ptr(), ldo,
        m, n, code, p, seed, sequence, offset, s), "ar_dropout")
    return out


def dropout_backward(dy, p: float, seed: int, sequence: int = 0, offset: int = 0, dx=None, stream=None):
    """Gradient of ``dropout`` with respect to x (that of ``residual`` is dy)."""
    code = _dropout_args(dy, seed, sequence, offset)
    lddy = _matrix(dy, "dy", dy.dtype, dy.device)
    m, n = dy.shape
    if dx is None:
        dx = torch.empty((m, n), dtype=dy.dtype, device=dy.device)
    lddx = _matrix(dx, "dx", dy.dtype, dy.device, m, n)
    lib = load()
    _launch(dy.device, stream, lambda s: lib.ar_dropout_backward(
        dy.data_ptr(), lddy, dx.data_ptr(), lddx, m, n, code, p, seed, sequence, offset, s),
        "ar_dropout_backward")
    return dx


def quantize_rows(x, q=None, scale=None, stream=None):
    """``(q, scale)``: ``scale[i] = max |x[i]| / 127``, ``q = rint(x / scale)`` in int8."""
    dev = _on_gpu(x, "x")
    code = _code(x.dtype, "x")
    ldx = _matrix(x, "x", x.dtype, dev)
    m, n = x.shape
    q = torch.empty((m, n), dtype=torch.int8, device=dev) if q is None else q
    scale = torch.empty(m, dtype=torch.float32, device=dev) if scale is None else scale
    ldq = _matrix(q, "q", torch.int8, dev, m, n)
    _vector(scale, "scale", m, dev)
    lib = load()
    _launch(dev, stream, lambda s: lib.ar_quantize_rows(
        x.data_ptr(), ldx, q.data_ptr(), ldq, scale.data_ptr(), m, n, code, s), "ar_quantize_rows")
    return q, scale


def _vector(t, what: str, n: int, device) -> None:
    if t.dtype != torch.float32 or t.device != device or t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be %d contiguous float32 values on %s" % (what, n, device))


def linear_i8(x, x_scale, w, w_scale, out=None, dtype=torch.bfloat16, stream=None):
    """``x_scale[m] * w_scale[n] * sum_k x[m, k] w[n, k]`` of int8 matrices, rounded to ``dtype``."""
    dev = _on_gpu(x, "x")
    ldx = _matrix(x, "x", torch.int8, dev)
    m, k = x.shape
    ldw = _matrix(w, "w", torch.int8, dev, None, k)
    n = w.shape[0]
    _vector(x_scale, "x_scale", m, dev)
    _vector(w_scale, "w_scale", n, dev)
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=dev)
    code = _code(out.dtype, "dtype", half=True)
    ldo = _matrix(out, "out", out.dtype, dev, m, n)
    lib = load()
    _launch(dev, stream, lambda s: lib.ar_linear_i8(
        x.data_ptr(), ldx, x_scale.data_ptr(), w.data_ptr(), ldw, w_scale.data_ptr(), out.data_ptr(), ldo,
        m, k, n, code, s), "ar_linear_i8")
    return out


def ops_device_status(stream=None) -> int:
    """AR_OK, or AR_ERR_TIMEOUT if a wait in one of these operators' kernels gave up (clears it)."""
    s = torch.cuda.current_stream() if stream is None else stream
    return load().ar_ops_get_device_status(s.cuda_stream)
