"""Argument checks of the 4-bit products at the C entry points, and the tests' own definitions; no GPU is touched."""
import ctypes

import pytest
import torch

from shot_allreduce_ranks_gb300 import _lib, build
from tests import layer_reference as layer

INVALID, UNSUPPORTED, OK = _lib.AR_ERR_INVALID_ARG, _lib.AR_ERR_UNSUPPORTED, _lib.AR_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("out,inner,group,want", [(16, 64, 64, (512, 16)), (17, 65, 64, (2048, 64)), (16, 64, 32, (512, 32)),
                                                  (16, 1, 128, (1024, 16)), (33, 257, 128, (9216, 144)), (1, 33, 32, (512, 32))])
def test_sizes(lib, out, inner, group, want):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.ar_i4_sizes(out, inner, group, ctypes.byref(a), ctypes.byref(b)) == OK
    assert (a.value, b.value) == want
    assert lib.ar_i4_sizes(out, inner, group, None, ctypes.byref(b)) == INVALID
    for bad in ((0, inner, group), (out, 0, group), (out, inner, 16), (out, inner, 256), (1 << 31, inner, group)):
        assert lib.ar_i4_sizes(*bad, ctypes.byref(a), ctypes.byref(b)) == INVALID


def refuses(f, base, kw, want, tail):
    a = dict(base)
    a.update(kw)
    assert f(*a.values(), *tail) == want


PACK = dict(q=16, ldq=96, scale=16, lds=3, zero=16, ldz=3, out=24, inner=96, group=32, data=16, ps=16, pz=16)


@pytest.mark.parametrize("kw", [dict(q=None), dict(ldq=95), dict(scale=None), dict(scale=17), dict(lds=2), dict(ldz=2), dict(zero=None),
                                dict(pz=None), dict(group=0), dict(out=0), dict(inner=0), dict(data=None), dict(data=24), dict(ps=None),
                                dict(ps=24), dict(pz=24)])
def test_pack_refuses(lib, kw):
    refuses(lib.ar_pack_i4, PACK, kw, INVALID, (None,))


QUANTIZE = dict(w=16, ldw=96, out=24, inner=96, group=32, dtype=0, data=16, ps=16, pz=None, scratch=16, bytes=24 * 3 * 3 + 24 * 96)


@pytest.mark.parametrize("kw,want", [(dict(w=None), INVALID), (dict(w=17), INVALID), (dict(ldw=95), INVALID), (dict(dtype=2), UNSUPPORTED),
                                     (dict(scratch=None), INVALID), (dict(bytes=24 * 9 + 24 * 96 - 1), INVALID), (dict(pz=17), INVALID)])
def test_quantize_refuses(lib, kw, want):
    refuses(lib.ar_quantize_i4, QUANTIZE, kw, want, (None,))
    assert lib.ar_quantize_i4_scratch_bytes(24, 96, 32) == QUANTIZE["bytes"] and lib.ar_quantize_i4_scratch_bytes(24, 96, 33) == 0


@pytest.mark.parametrize("kw,want", [(dict(data=None), INVALID), (dict(ps=17), INVALID), (dict(w=None), INVALID), (dict(ldw=95), INVALID),
                                     (dict(dtype=2), UNSUPPORTED), (dict(group=1), INVALID)])
def test_dequantize_refuses(lib, kw, want):
    refuses(lib.ar_dequantize_i4, dict(data=16, ps=16, pz=None, out=24, inner=96, group=32, dtype=0, w=16, ldw=96), kw, want, (None,))


@pytest.mark.parametrize("kw,want", [(dict(x=None), INVALID), (dict(x=17), INVALID), (dict(ldx=95), INVALID), (dict(data=None), INVALID),
                                     (dict(ps=None), INVALID), (dict(pz=18), INVALID), (dict(y=None), INVALID), (dict(y=17), INVALID),
                                     (dict(ldy=23), INVALID), (dict(inner=0), INVALID), (dict(out=0), INVALID), (dict(group=96), INVALID),
                                     (dict(dtype=2), UNSUPPORTED), (dict(tokens=32 * 65535 + 1), INVALID),
                                     (dict(tokens=0, x=None, data=None, y=None), OK)])
def test_linear_refuses(lib, kw, want):
    base = dict(x=16, ldx=96, data=16, ps=16, pz=None, y=16, ldy=24, tokens=5, inner=96, out=24, group=32, dtype=0)
    refuses(lib.ar_linear_i4, base, kw, want, (None,))


@pytest.mark.parametrize("zero", [False, True])
def test_the_definition_of_the_quantisation(zero):
    g = torch.Generator().manual_seed(1)
    w = torch.randn(5, 70, generator=g).bfloat16()
    q, scale, z = layer.quantize_i4(w, 32, zero)
    assert int(q.max()) <= 15 and (zero or int(q.min()) >= 1) and scale.shape == (5, 3)
    step = scale.double().repeat_interleave(32, 1)[:, :70]
    off = (layer.weights_i4(q, scale, z, 32) - w.double()).abs()
    # the scale's rounding moves the ends by up to 7 or 15 of its 2^-8
    assert bool((off <= step * ((1.0 if zero else 0.5) + 15 * 2.0 ** -8)).all())
