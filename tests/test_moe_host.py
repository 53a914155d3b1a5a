"""Argument checks of the layer of experts at the C entry points; no GPU is touched."""
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


DESCRIPTION = dict(dtype=0, logits_dtype=2, activation=0, experts=8, first_expert=2, local_experts=4, top_k=3, normalize=1, hidden=16, width=12)
CALL = dict(x=16, ldx=16, logits=16, ldl=8, wg=16, wu=16, ldw=16, esw=192, wd=16, ldd=12, esd=192, out=16, ldo=16, expert=16,
            weight=16, tokens=5, scratch=16, bytes=480 + 16 + 160 * 2 * 32 * 16 * 4)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(logits_dtype=3), UNSUPPORTED), (dict(activation=2), INVALID),
    (dict(experts=0), INVALID), (dict(experts=1025), INVALID), (dict(first_expert=-1), INVALID), (dict(first_expert=5), INVALID),
    (dict(local_experts=0), INVALID), (dict(local_experts=9), INVALID), (dict(top_k=0), INVALID), (dict(top_k=9), INVALID),
    (dict(experts=100, top_k=17), INVALID), (dict(hidden=0), INVALID), (dict(width=0), INVALID), (dict(width=1 << 31), INVALID),
    (dict(x=None), INVALID), (dict(x=17), INVALID), (dict(ldx=15), INVALID), (dict(logits=None), INVALID), (dict(logits=18), INVALID),
    (dict(ldl=7), INVALID), (dict(wg=None), INVALID), (dict(wu=17), INVALID), (dict(ldw=15), INVALID), (dict(wd=None), INVALID),
    (dict(ldd=11), INVALID), (dict(esd=1 << 41), INVALID), (dict(out=None), INVALID), (dict(out=17), INVALID), (dict(ldo=15), INVALID),
    (dict(expert=18), INVALID), (dict(weight=18), INVALID), (dict(scratch=None), INVALID), (dict(scratch=24), INVALID),
    (dict(bytes=480 + 15 + 160 * 4096), INVALID), (dict(tokens=0, x=None, out=None, scratch=None), OK)])
def test_refuses(lib, kw, want):
    d, a = dict(DESCRIPTION), dict(CALL)
    for k, v in kw.items():
        (d if k in d else a)[k] = v
    assert lib.ar_moe_ffn(ctypes.byref(_lib.ArMoe(*d.values())), *a.values(), None) == want
    assert lib.ar_moe_ffn(None, *a.values(), None) == INVALID


def test_scratch_bytes(lib):
    def f(tokens, **k):
        return lib.ar_moe_scratch_bytes(ctypes.byref(_lib.ArMoe(*dict(DESCRIPTION, **k).values())), tokens)

    # the experts' inner rows, a count for every 16 columns of the result, and what is left of them in parts
    parts = 160 * 2 * 32 * 16 * 4
    assert f(5) == 480 + 16 + parts and f(1000) == 32 * 3 * 16 * 2 + 16 + parts and f(0) == 0
    assert f(5, width=17) == 5 * 3 * 24 * 2 + 16 + parts and f(5, hidden=81) == 480 + 32 + parts
    assert f(5, top_k=9) == 0 and lib.ar_moe_scratch_bytes(None, 5) == 0


def test_the_definition_of_the_routing():
    inf = float("inf")
    z = torch.tensor([[1.0, 3.0, 3.0, 0.0], [-inf, -inf, 2.0, -inf], [-inf] * 4, [0.0, float("nan"), 5.0, inf]])
    e, w, _ = layer.routing(z, 2, True)
    assert e.tolist() == [[1, 2], [2, -1], [-1, -1], [1, 3]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [0.0, 0.0]
    assert torch.isnan(w[3]).all()
    p = torch.softmax(z[0].double(), 0)
    assert torch.allclose(layer.routing(z, 2, False)[1][0], p[[1, 2]])
