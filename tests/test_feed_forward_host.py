"""The feed-forward operators' argument checks, at the C entry points and in
the Python binding, and the tests' own generator against published vectors;
no GPU is touched."""
import ctypes

import numpy as np
import pytest
import torch

from shot_allreduce_ranks_gb300 import _lib, build
from tests import ff_reference as ref

INVALID, UNSUPPORTED, OK = _lib.AR_ERR_INVALID_ARG, _lib.AR_ERR_UNSUPPORTED, _lib.AR_OK
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("args,want", [
    ((0, 8, 8, 0, 0, 0), INVALID), ((8, 0, 8, 0, 0, 0), INVALID), ((8, 8, 0, 0, 0, 0), INVALID),
    ((8, 8, 8, 0, 2, 0), INVALID), ((8, 8, 8, 0, -1, 0), INVALID), ((BIG, 8, 8, 0, 0, 0), INVALID),
    ((8, 8, 8, _lib.AR_FP32, 0, 0), UNSUPPORTED), ((8, 8, 8, 7, 0, 0), UNSUPPORTED)])
def test_ffn_create_refuses(lib, args, want):
    h = ctypes.c_void_p(1)
    assert lib.ar_ffn_create(*args, ctypes.byref(h)) == want
    assert h.value is None
    assert lib.ar_ffn_create(*args, None) == INVALID


def test_ffn_calls_without_a_handle(lib):
    assert lib.ar_ffn_forward(None, 16, 8, 16, 16, 8, 16, None, None, 8, 1, None, 0, None) == INVALID
    assert lib.ar_ffn_backward(None, 16, 8, 16, 16, 8, 16, 16, 16, 8, 16, 8, 16, 16, 8, 1, None, 0, None) == INVALID
    assert lib.ar_ffn_scratch_bytes(None, 16, 8, 16, 16, 8, 1) == 0
    assert lib.ar_ffn_destroy(None) == OK


def dropout_args(**kw):
    a = dict(x=16, ldx=8, res=None, ldr=0, out=32, ldo=8, rows=2, cols=8, dtype=0, p=0.5, seed=1,
             sequence=0, offset=0)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), UNSUPPORTED), (dict(p=-0.1), INVALID), (dict(p=1.5), INVALID),
    (dict(p=float("nan")), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(ldx=7), INVALID), (dict(ldo=7), INVALID), (dict(res=64, ldr=7), INVALID),
    (dict(x=17), INVALID), (dict(out=33), INVALID), (dict(dtype=2, x=18), INVALID),
    (dict(offset=2 ** 64 - 8), INVALID), (dict(rows=BIG), INVALID),
    (dict(rows=1 << 38, cols=1 << 38, ldx=1 << 38, ldo=1 << 38), INVALID),
    (dict(rows=0, x=None, out=None), OK), (dict(cols=0), OK)])
def test_dropout_refuses(lib, kw, want):
    a = dropout_args(**kw)
    assert lib.ar_dropout(*a, None) == want
    if "res" not in kw:
        assert lib.ar_dropout_backward(*(a[:2] + a[4:]), None) == want


@pytest.mark.parametrize("args,want", [
    ((16, 8, 16, 8, 16, 2, 8, 3), UNSUPPORTED), ((None, 8, 16, 8, 16, 2, 8, 0), INVALID),
    ((16, 8, None, 8, 16, 2, 8, 0), INVALID), ((16, 8, 16, 8, None, 2, 8, 0), INVALID),
    ((16, 7, 16, 8, 16, 2, 8, 0), INVALID), ((16, 8, 16, 7, 16, 2, 8, 0), INVALID),
    ((16, 8, 16, 8, 16, 2, 0, 0), INVALID), ((17, 8, 16, 8, 16, 2, 8, 0), INVALID),
    ((16, 8, 16, 8, 18, 2, 8, 0), INVALID), ((16, 8, 16, 8, 16, 0, 8, 0), OK)])
def test_quantize_rows_refuses(lib, args, want):
    assert lib.ar_quantize_rows(*args, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(x=None), INVALID), (dict(ldx=7), INVALID), (dict(sx=None), INVALID), (dict(sx=18), INVALID),
    (dict(w=None), INVALID), (dict(ldw=7), INVALID), (dict(sw=None), INVALID), (dict(y=None), INVALID),
    (dict(ldy=3), INVALID), (dict(y=17), INVALID), (dict(k=0), INVALID), (dict(n=0), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(m=0), OK)])
def test_linear_i8_refuses(lib, change, want):
    a = dict(x=16, ldx=8, sx=16, w=16, ldw=8, sw=16, y=16, ldy=4, m=2, k=8, n=4, dtype=0)
    a.update(change)
    assert lib.ar_linear_i8(*a.values(), None, 0, None) == want


def test_linear_i8_scratch_bytes(lib):
    """Only rows that do not start on 16 bytes are counted, each rounded up to 128."""
    f = lib.ar_linear_i8_scratch_bytes
    assert f(16, 32, 32, 32, 50, 32, 7) == 0
    assert f(17, 32, 32, 32, 50, 32, 7) == 50 * 128
    assert f(16, 133, 32, 133, 50, 133, 7) == (50 + 7) * 256
    assert f(16, 32, 33, 32, 50, 20, 7) == 7 * 128
    assert f(17, 33, 33, 33, 32, 20, 7) == 0  # few tokens are read where they are


def test_python_refuses_what_is_not_on_a_gpu():
    import shot_allreduce_ranks_gb300 as ar
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ar.dropout(x, 0.5, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ar.quantize_rows(x)
    with pytest.raises(ValueError, match="CUDA"):
        ar.linear_i8(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4))
    with pytest.raises(ValueError, match="activation"):
        ar.GatedFFN(4, 8, 8, activation="relu")
    with pytest.raises(ValueError, match="dtype"):
        ar.GatedFFN(4, 8, 8, dtype=torch.float32)
    with pytest.raises(ValueError, match="at least 1"):
        ar.GatedFFN(0, 8, 8)


@pytest.mark.parametrize("counter,key,want", [
    # The generator's published known answers: all zeros, all ones.
    ((0, 0), 0, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    (((1 << 64) - 1, (1 << 64) - 1), (1 << 64) - 1, "408f276d 41c83b0e a20bc7c6 6d5451fd")])
def test_the_generator_of_the_tests(counter, key, want):
    block, sequence = counter
    got = ref.draws(block * 4, 4, key, sequence)
    assert " ".join("%08x" % v for v in got) == want


def test_gradient_formula_against_differences():
    """The 64-bit gradient that the kernels are held to, against central differences of the 64-bit forward pass."""
    gen = torch.Generator().manual_seed(3)
    for act in ("silu", "gelu"):
        x, wg, wu = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((3, 5), (4, 5), (4, 5)))
        dout = torch.randn(3, 4, generator=gen, dtype=torch.float64)

        def loss(x, wg, wu):
            g = x @ wg.T
            return float((ref.activation(g, act)[0] * (x @ wu.T) * dout).sum())

        f, df, _, _ = ref.activation(x @ wg.T, act)
        a, b = dout * (x @ wu.T) * df, dout * f
        for k, grad in enumerate((a @ wg + b @ wu, a.T @ x, b.T @ x)):
            for i in np.ndindex(*grad.shape):
                t = [x, wg, wu]
                up, down = t[k].clone(), t[k].clone()
                up[i] += 1e-5
                down[i] -= 1e-5
                d = (loss(*t[:k], up, *t[k + 1:]) - loss(*t[:k], down, *t[k + 1:])) / 2e-5
                # truncation ~ h^2 f''' ~ 1e-9, rounding ~ 1e-16 / 1e-5 * |loss| ~ 1e-9
                assert abs(d - float(grad[i])) < 1e-7
