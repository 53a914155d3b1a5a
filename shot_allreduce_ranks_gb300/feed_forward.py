"""Feed-forward operators around the sum over ranks (contracts in include/ar.h).

``GatedFFN`` is one rank's shard of the gated projections with its gradients,
``linear_i8`` (with ``quantize_rows``) the down projection in 8-bit integers,
``dropout`` the step after the sum, its mask drawn from the elements' places
and never stored.  Matrices are 2-D CUDA tensors whose rows are contiguous
(any row stride).  Calls are asynchronous on the current (or given) stream of
the tensors' device, which also owns the outputs that a call allocates; a
given stream of another device is refused.  torch's differentiation does not
record them: the backward passes are calls of their own, and a forward pass
warns where an input requires grad (not under ``torch.no_grad()``).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from ._lib import ACTIVATIONS, AR_BF16, AR_FP16, AR_FP32, PKG, check, load

_CODES = {torch.bfloat16: AR_BF16, torch.float16: AR_FP16, torch.float32: AR_FP32}


def _load_ops():
    """The compiled binding (checks, allocation of outputs, the C calls)."""
    path = os.path.join(PKG, "_ops.so")
    if not os.path.exists(path):
        raise RuntimeError("_ops.so is not built (%s); run `python -m shot_allreduce_ranks_gb300.build`" % path)
    load()
    spec = importlib.util.spec_from_file_location(__package__ + "._ops", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.set_check(check)
    return module


class _NotLoaded:
    """Stands for the binding until its first call, so that importing names needs no built library."""

    def __getattr__(self, name):
        global _ops
        _ops = _load_ops()
        return getattr(_ops, name)


_ops = _NotLoaded()


def _current(stream, device):
    """The context in which `stream` is the current one of `device`, which it has to belong to."""
    if device is not None and stream.device != device:
        raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, device))
    return torch.cuda.stream(stream)


# Freeing a workspace waits for the device, which ends a capture with an error.
# Handles that are collected during one wait here for the next handle that is made or closed.
_late = []


def _capturing(device) -> bool:
    """Whether the device's current stream is being captured into a graph."""
    if torch.cuda.current_device() == device.index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(device):
        return torch.cuda.is_current_stream_capturing()


def _destroy(h, device) -> None:
    with torch.cuda.device(device):
        check(load().ar_ffn_destroy(h), "ar_ffn_destroy")


def _destroy_late() -> None:
    while _late and not _capturing(_late[-1][1]):
        _destroy(*_late.pop())


class GatedFFN:
    """One rank's gated feed-forward shard: ``act(x Wgate^T) * (x Wup^T)``.

    ``hidden`` is the width of x, ``width`` this rank's rows of both weight
    matrices.  ``train=True`` also allocates the workspace of ``backward`` for
    up to ``max_tokens`` rows; without it ``backward`` is refused.
    ``backward`` calls share that workspace: order them on one stream.  Freeing
    it waits for the device: ``close`` is refused while a graph is being
    captured, and a handle that is collected then is freed later.  A graph that
    holds a ``backward`` holds the workspace's address: such a handle
    (``captured``) is freed by ``close`` alone, to be called when no such graph
    is replayed any more, and not by being collected.
    """

    captured = False

    def __init__(self, max_tokens: int, hidden: int, width: int, dtype=torch.bfloat16,
                 activation: str = "silu", train: bool = False, device=None):
        if activation not in ACTIVATIONS:
            raise ValueError("activation must be one of %s" % ", ".join(sorted(ACTIVATIONS)))
        self.max_tokens, self.hidden, self.width = int(max_tokens), int(hidden), int(width)
        self.dtype, self.train = dtype, bool(train)
        if min(self.max_tokens, self.hidden, self.width) < 1:
            raise ValueError("max_tokens, hidden and width must be at least 1")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be torch.bfloat16 or torch.float16, got %s" % dtype)
        index = None if device is None else torch.device(device).index
        self.device = torch.device("cuda", torch.cuda.current_device() if index is None else index)
        _destroy_late()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(load().ar_ffn_create(self.max_tokens, self.hidden, self.width, _CODES[dtype],
                                       ACTIVATIONS[activation], int(self.train), ctypes.byref(h)),
                  "ar_ffn_create")
        self._h = h
        self._constants = (h.value, _CODES[dtype], self.hidden, self.width, self.device.index, self.max_tokens)

    def close(self) -> None:
        if getattr(self, "_h", None):
            if self.train and _capturing(self.device):
                raise RuntimeError("a GatedFFN with a workspace is not closed while a graph is being captured")
            h, self._h, self._constants = self._h, None, None
            _destroy(h, self.device)
            _destroy_late()

    def __del__(self):
        try:
            if self.captured:
                return
            if self.train and self._h and _capturing(self.device):
                _late.append((self._h, self.device))
            else:
                self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def forward(self, x, w_gate, w_up, out=None, gate=None, up=None, save: bool = False, stream=None):
        """``out``; with ``save`` (or given ``gate`` and ``up``) ``(out, gate, up)``."""
        if stream is not None:
            with _current(stream, self.device):
                return self.forward(x, w_gate, w_up, out, gate, up, save)
        return _ops.ffn_forward(self._constants, x, w_gate, w_up, out, gate, up, save)

    def backward(self, x, w_gate, w_up, gate, up, dout, dx=None, dw_gate=None, dw_up=None,
                 need_dx: bool = True, need_dw: bool = True, stream=None):
        """``(dx, dw_gate, dw_up)`` from the saved ``gate`` and ``up``; None for what is not needed."""
        if stream is not None:
            with _current(stream, self.device):
                return self.backward(x, w_gate, w_up, gate, up, dout, dx, dw_gate, dw_up, need_dx, need_dw)
        if not self.captured and _capturing(self.device):
            self.captured = True
        return _ops.ffn_backward(self._constants, x, w_gate, w_up, gate, up, dout, dx, dw_gate, dw_up, need_dx,
                                 need_dw)


def dropout(x, p: float, seed: int, sequence: int = 0, offset: int = 0, residual=None, out=None,
            stream=None):
    """``residual + (keep ? x / (1 - p) : 0)``, the mask drawn from each element's place.

    Element (i, j) draws at ``offset + i * cols + j`` of the stream that
    ``seed`` and ``sequence`` name; equal arguments draw equal masks.
    """
    if stream is not None:
        with _current(stream, getattr(x, "device", None)):
            return _ops.dropout(x, p, seed, sequence, offset, residual, out)
    return _ops.dropout(x, p, seed, sequence, offset, residual, out)


def dropout_backward(dy, p: float, seed: int, sequence: int = 0, offset: int = 0, dx=None, stream=None):
    """Gradient of ``dropout`` with respect to x (that of ``residual`` is dy)."""
    if stream is not None:
        with _current(stream, getattr(dy, "device", None)):
            return _ops.dropout_backward(dy, p, seed, sequence, offset, dx)
    return _ops.dropout_backward(dy, p, seed, sequence, offset, dx)


def quantize_rows(x, q=None, scale=None, stream=None):
    """``(q, scale)``: ``scale[i] = max |x[i]| / 127``, ``q = rint(x / scale)`` in int8.

    The rows of a new ``q`` start on 16 bytes, so that ``linear_i8`` reads them as they are.
    """
    if stream is not None:
        with _current(stream, getattr(x, "device", None)):
            return _ops.quantize_rows(x, q, scale)
    return _ops.quantize_rows(x, q, scale)


def linear_i8(x, x_scale, w, w_scale, out=None, dtype=torch.bfloat16, stream=None):
    """``x_scale[m] * w_scale[n] * sum_k x[m, k] w[n, k]`` of int8 matrices, rounded to ``dtype``."""
    code = _CODES.get(dtype)
    if code is None or code == AR_FP32:
        raise ValueError("dtype must be torch.bfloat16 or torch.float16, got %s" % dtype)
    if stream is not None:
        with _current(stream, getattr(x, "device", None)):
            return _ops.linear_i8(x, x_scale, w, w_scale, out, code)
    return _ops.linear_i8(x, x_scale, w, w_scale, out, code)


def ops_device_status(stream=None) -> int:
    """AR_OK, or AR_ERR_TIMEOUT if a wait in one of these operators' kernels gave up (clears it).

    Read on the device of the given stream, or of the current one.
    """
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        return load().ar_ops_get_device_status(s.cuda_stream)
