"""Feed-forward operators around the sum over ranks (contracts in include/ar.h).

``GatedFFN`` is one rank's shard of the gated projections with its gradients,
``linear_i8`` (with ``quantize_rows``) the down projection in 8-bit integers,
``dropout`` the step after the sum, its mask drawn from the elements' places
and never stored; ``residual_norm`` the norms before and after a block with its
gate and the residual, ``linear_i4`` products of a few tokens with 4-bit weights,
``moe_ffn`` a layer of gated experts for a few tokens.  Matrices are 2-D CUDA tensors whose rows are contiguous
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

from ._lib import ACTIVATIONS, AR_BF16, AR_FP16, AR_FP32, NORMS, PKG, check, load

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


class Int4Weight:
    """A matrix of 4-bit weights as ``linear_i4`` reads it: made by ``pack_i4`` or ``quantize_i4``.

    ``shape`` is that of the matrix, ``dtype`` that of the scales and of the
    activations that it multiplies.  ``data``, ``scale`` and ``zero`` (or None) are the
    laid-out arrays; their order is the library's own.
    """

    def __init__(self, data, scale, zero, shape, group: int):
        self.data, self.scale, self.zero = data, scale, zero
        self.shape, self.group, self.dtype, self.device = tuple(shape), int(group), scale.dtype, data.device
        self._constants = (data, scale, zero, *self.shape, self.group)

    def dequantize(self, out=None, stream=None):
        """The matrix that the weights stand for, rounded to ``dtype`` (for a product of many tokens)."""
        if stream is not None:
            with _current(stream, self.device):
                return _ops.dequantize_i4(self._constants, out)
        return _ops.dequantize_i4(self._constants, out)

    def __repr__(self):
        return "Int4Weight(%d x %d, group=%d, dtype=%s, zero=%s)" % (*self.shape, self.group, self.dtype, self.zero is not None)


def pack_i4(q, scale, zero=None, group: int = 128, stream=None) -> Int4Weight:
    """Lays out 4-bit weights: ``scale[n, k // group] * (q[n, k] - zero[n, k // group])``.

    ``q`` and ``zero`` are uint8 matrices of which the low four bits count, zero 8 where it
    is None; ``scale`` is in bfloat16 or float16.  ``group`` is 32, 64 or 128.
    """
    if stream is not None:
        with _current(stream, getattr(q, "device", None)):
            return pack_i4(q, scale, zero, group)
    return Int4Weight(*_ops.pack_i4(q, scale, zero, group), q.shape, group)


def quantize_i4(w, group: int = 128, zero: bool = False, stream=None) -> Int4Weight:
    """A matrix of weights in 4 bits, each group of a row by itself: symmetric, or with zero points."""
    if stream is not None:
        with _current(stream, getattr(w, "device", None)):
            return quantize_i4(w, group, zero)
    return Int4Weight(*_ops.quantize_i4(w, group, zero), w.shape, group)


def linear_i4(x, weight: Int4Weight, out=None, stream=None):
    """``x W^T`` with 4-bit weights, for a few tokens: the weights are read once for every 32 rows of x."""
    if not isinstance(weight, Int4Weight):
        raise TypeError("weight must be an Int4Weight, got %s" % type(weight).__name__)
    if stream is not None:
        with _current(stream, getattr(x, "device", None)):
            return _ops.linear_i4(x, weight._constants, out)
    return _ops.linear_i4(x, weight._constants, out)


def moe_ffn(x, logits, w_gate, w_up, w_down, top_k: int, activation: str = "silu", normalize: bool = True,
            first_expert: int = 0, out=None, routing: bool = False, stream=None):
    """A layer of gated experts for a few tokens; with ``routing`` ``(out, expert, weight)``.

    Token t goes to the experts of its ``top_k`` highest ``logits`` (equal ones by the
    lowest index), weighted by their softmax over all experts or, with
    ``normalize``, over the chosen ones::

        out[t] = sum_j weight[t, j] * ((act(x[t] Wgate_e^T) * (x[t] Wup_e^T)) Wdown_e^T),   e = expert[t, j]

    ``w_gate`` and ``w_up`` are experts x width x hidden, ``w_down`` experts x
    hidden x width.  They may be a part of the layer's experts, from
    ``first_expert`` on, or of their width: the ranks' outputs are then summed.  A logit of
    -infinity is never chosen (expert -1, weight 0, where fewer remain).  What is between the
    two products is held as the sum of two numbers of x's type, so that its rounding does not show
    (in float16 it becomes an infinity from 65,520 on).  Each matrix in use is read once for every 32 tokens.
    """
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be one of %s" % ", ".join(sorted(ACTIVATIONS)))
    if stream is not None:
        with _current(stream, getattr(x, "device", None)):
            return _ops.moe_ffn(x, logits, w_gate, w_up, w_down, top_k, ACTIVATIONS[activation], normalize, first_expert,
                                out, routing)
    return _ops.moe_ffn(x, logits, w_gate, w_up, w_down, top_k, ACTIVATIONS[activation], normalize, first_expert, out,
                        routing)


def _kind(kind: str) -> int:
    if kind not in NORMS:
        raise ValueError("kind must be one of %s" % ", ".join(sorted(NORMS)))
    return NORMS[kind]


def residual_norm(x, residual=None, weight=None, bias=None, after_weight=None, after_bias=None, gate=None,
                  kind: str = "rms", eps: float = 1e-6, residual_scale: float = 1.0, weight_offset: float = 0.0,
                  r=None, y=None, stream=None):
    """``(r, y)``: the norm after a block, its gate, the residual and the norm before the next block, in one pass.

    With ``norm(v)`` the rows over the root of their mean square (``kind="rms"``),
    or less their mean over their standard deviation (``"layer"``)::

        z = norm(x) * (weight_offset + after_weight) + after_bias      x itself without after_weight
        r = residual_scale * residual + gate * z
        y = norm(r) * (weight_offset + weight) + bias                  None without weight

    ``gate`` is a matrix whose row g is for the rows / gate rows rows from
    g * rows / gate rows on: one row for all, one a sequence, or one a token.
    Without residual, gate and after_weight r would be x and None is
    returned for it.  ``r`` and ``y`` may be given, and be x and the residual (either way).
    """
    k = _kind(kind)
    if stream is not None:
        with _current(stream, getattr(x, "device", None)):
            return _ops.residual_norm(x, residual, weight, bias, after_weight, after_bias, gate, k, eps, residual_scale,
                                      weight_offset, r, y)
    return _ops.residual_norm(x, residual, weight, bias, after_weight, after_bias, gate, k, eps, residual_scale,
                              weight_offset, r, y)


def residual_norm_backward(dy, dr, x, r, weight=None, bias=None, after_weight=None, after_bias=None, gate=None,
                           kind: str = "rms", eps: float = 1e-6, residual_scale: float = 1.0,
                           weight_offset: float = 0.0, need_dresidual: bool = True, stream=None):
    """``(dx, dresidual, dweight, dbias, dafter_weight, dafter_bias, dgate)`` from the gradients of y and r.

    ``dr`` None counts as 0; ``dy`` is None where there was no weight.  ``x`` and
    ``r`` are the forward pass's: x may be None without gate and after_weight, r
    is None where the forward pass gave None.  A weight, bias or gate that was not given has None for its gradient;
    dresidual is None without r and where ``need_dresidual`` is False (the call cannot see whether there was a
    residual: without one, say so, and a matrix is not written).  Where neither a gate, nor
    after_weight, nor a scale stands between them, dx and dresidual are equal and one
    tensor is returned for both.
    """
    k = _kind(kind)
    if stream is not None:
        with _current(stream, getattr(dr if dy is None else dy, "device", None)):
            return _ops.residual_norm_backward(dy, dr, x, r, weight, bias, after_weight, after_bias, gate, k, eps,
                                               residual_scale, weight_offset, need_dresidual)
    return _ops.residual_norm_backward(dy, dr, x, r, weight, bias, after_weight, after_bias, gate, k, eps,
                                       residual_scale, weight_offset, need_dresidual)


def ops_device_status(stream=None) -> int:
    """AR_OK, or AR_ERR_TIMEOUT if a wait in one of these operators' kernels gave up (clears it).

    Read on the device of the given stream, or of the current one.
    """
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        return load().ar_ops_get_device_status(s.cuda_stream)
