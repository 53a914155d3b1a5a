"""Argument checks of the norms at the C entry points, and the tests' own formulas; no GPU is touched."""
import ctypes

import numpy as np
import pytest
import torch

from shot_allreduce_ranks_gb300 import _lib, build
from tests import layer_reference as layer

INVALID, UNSUPPORTED, OK = _lib.AR_ERR_INVALID_ARG, _lib.AR_ERR_UNSUPPORTED, _lib.AR_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def description(kind=0, dtype=0, rows=4, cols=8, gate_rows=0, eps=1e-6, **_):
    return _lib.ArNorm(kind, dtype, rows, cols, gate_rows, eps, 1.0, 0.0)


FORWARD = dict(x=16, ldx=8, res=None, ldres=0, gate=None, ldg=0, aw=None, ab=None, w=32, b=None, r=64, ldr=8, y=96, ldy=8)
COMMON = [
    (dict(kind=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(cols=0), INVALID),
    (dict(cols=(1 << 30) + 1), INVALID), (dict(rows=(1 << 40) + 1), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(ab=16), INVALID), (dict(w=33), INVALID),
    (dict(gate=16, ldg=8), INVALID), (dict(gate_rows=2), INVALID), (dict(gate=16, ldg=8, gate_rows=3), INVALID),
    (dict(gate=16, ldg=7, gate_rows=2), INVALID), (dict(gate=17, ldg=8, gate_rows=2), INVALID)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(x=None), INVALID), (dict(ldx=7), INVALID), (dict(x=17), INVALID), (dict(y=None), INVALID), (dict(ldy=7), INVALID),
    (dict(w=None, y=None), INVALID), (dict(w=None, aw=32), INVALID), (dict(ldr=7), INVALID), (dict(r=65), INVALID),
    (dict(res=16, ldres=7), INVALID), (dict(res=17, ldres=8), INVALID), (dict(b=33), INVALID),
    (dict(w=None, aw=32, y=None, b=32), INVALID), (dict(dtype=2, x=18), INVALID),
    (dict(w=None, aw=32, y=None, r=None), OK), (dict(rows=0, x=None, r=None), OK)])
def test_forward_refuses(lib, kw, want):
    a = dict(FORWARD)
    a.update({k: v for k, v in kw.items() if k in a})
    assert lib.ar_residual_norm(ctypes.byref(description(**kw)), *a.values(), None) == want


def test_a_description_is_needed(lib):
    assert lib.ar_residual_norm(None, *FORWARD.values(), None) == INVALID


BACKWARD = dict(dy=16, lddy=8, dr=16, lddr=8, x=16, ldx=8, r=16, ldr=8, gate=None, ldg=0, aw=None, ab=None, w=32, dx=64,
                lddx=8, dres=64, lddres=8, dgate=None, lddg=0, dw=64, db=None, daw=None, dab=None, scratch=64, bytes=128)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(dy=None), INVALID), (dict(r=None), INVALID), (dict(lddy=7), INVALID), (dict(ldr=7), INVALID), (dict(lddr=7), INVALID),
    (dict(lddx=7), INVALID), (dict(lddres=7), INVALID), (dict(dx=65), INVALID), (dict(dgate=64, lddg=8), INVALID),
    (dict(daw=64), INVALID), (dict(w=None, aw=32), INVALID), (dict(scratch=None), INVALID), (dict(scratch=68), INVALID),
    (dict(bytes=127), INVALID), (dict(gate=16, ldg=8, gate_rows=2, x=None), INVALID), (dict(dw=65), INVALID),
    (dict(gate=16, ldg=8, gate_rows=2, dgate=64, lddg=7), INVALID), (dict(aw=32, x=None), INVALID),
    (dict(w=None, dy=None, dw=None, aw=32, dr=None), INVALID), (dict(dx=None, dres=None, dw=None), OK)])
def test_backward_refuses(lib, kw, want):
    a = dict(BACKWARD)
    a.update({k: v for k, v in kw.items() if k in a})
    assert lib.ar_residual_norm_backward(ctypes.byref(description(**kw)), *a.values(), None) == want


def test_scratch_bytes(lib):
    f = lib.ar_residual_norm_scratch_bytes
    assert f(4, 8, 0) == 0 and f(4, 8, 1) == 128 and f(0, 8, 3) == 0
    # a row of parts for every CTA, of which there are no more than rows
    assert f(10 ** 6, 100, 5) == 5 * 640 * 400 and f(10 ** 6, 8192, 1) == 320 * 8192 * 4 and f(100, 20000, 2) == 2 * 100 * 80000


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gates", [0, 1, 3, 6])
def test_gradient_formulas_against_differences(kind, gates):
    """The 64-bit gradients that the kernels are held to, against central differences of the 64-bit forward pass."""
    g = torch.Generator().manual_seed(gates)
    rows, cols = 6, 5

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64)

    a = dict(x=normal(rows, cols), residual=normal(rows, cols), weight=normal(cols), bias=normal(cols),
             after_weight=normal(cols), after_bias=normal(cols))
    if gates:
        a["gate"] = normal(gates, cols)
    dy, dr = normal(rows, cols), normal(rows, cols)
    more = dict(kind=kind, eps=1e-3, residual_scale=0.6, weight_offset=0.25)

    def loss(values):
        (r, _), (y, _) = layer.Norm(**values, **more).forward()
        return float((r * dr).sum() + (y * dy).sum())

    (r, _), _ = layer.Norm(**a, **more).forward()
    got = layer.Norm(**a, **more).backward(dy, dr, r)
    assert set(got) == {"d" + k for k in a}
    for k, v in a.items():
        for i in np.ndindex(*v.shape):
            up, down = v.clone(), v.clone()
            up[i] += 1e-5
            down[i] -= 1e-5
            d = (loss(dict(a, **{k: up})) - loss(dict(a, **{k: down}))) / 2e-5
            # truncation ~ h^2 f''' / 6, f''' up to 1e3 here, rounding ~ 1e-16 |loss| / 1e-5
            assert abs(d - float(got["d" + k][0][i])) < 1e-6 * (1 + abs(d))
