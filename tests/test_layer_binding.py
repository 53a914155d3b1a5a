"""The layer operators' Python face with stand-ins for the GPU's side: streams of another device, arguments in order."""
from types import SimpleNamespace

import pytest
import torch

from shot_allreduce_ranks_gb300 import build


@pytest.fixture(scope="module")
def ff():
    build.build()
    from shot_allreduce_ranks_gb300 import feed_forward
    return feed_forward


def on(index):
    return SimpleNamespace(device=torch.device("cuda", index), cuda_stream=70 + index)


def packed(ff, index=0):
    return ff.Int4Weight(SimpleNamespace(device=torch.device("cuda", index)), SimpleNamespace(dtype=torch.bfloat16), None, (8, 64), 32)


def test_a_stream_of_another_device_is_refused(ff, monkeypatch):
    def used(stream):
        raise AssertionError("the stream was used")

    monkeypatch.setattr(torch.cuda, "stream", used)
    x, s = on(0), on(1)
    for call in (lambda: ff.residual_norm(x, weight=x, stream=s), lambda: ff.residual_norm_backward(x, None, x, None, x, stream=s),
                 lambda: ff.residual_norm_backward(None, x, x, x, after_weight=x, stream=s), lambda: ff.pack_i4(x, x, stream=s),
                 lambda: ff.quantize_i4(x, stream=s), lambda: ff.linear_i4(x, packed(ff), stream=s),
                 lambda: packed(ff).dequantize(stream=s), lambda: ff.moe_ffn(x, x, x, x, x, 1, stream=s)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_what_reaches_the_binding(ff, monkeypatch):
    """Names and places of the arguments, by a binding that returns them."""
    class Echo:
        def __getattr__(self, name):
            return lambda *a: (name, *a)

    monkeypatch.setattr(ff, "_ops", Echo())
    assert ff.residual_norm(1, 2, 3, 4, 5, 6, 7, kind="layer", eps=8.0, residual_scale=9.0, weight_offset=10.0, r=11, y=12) == \
        ("residual_norm", 1, 2, 3, 4, 5, 6, 7, 1, 8.0, 9.0, 10.0, 11, 12)
    assert ff.residual_norm_backward(1, 2, 3, 4, 5, 6, 7, 8, 9, eps=0.5, residual_scale=2.0, weight_offset=3.0, need_dresidual=False) == \
        ("residual_norm_backward", 1, 2, 3, 4, 5, 6, 7, 8, 9, 0, 0.5, 2.0, 3.0, False)
    assert ff.moe_ffn(1, 2, 3, 4, 5, 6, activation="gelu", normalize=False, first_expert=7, out=8, routing=True) == \
        ("moe_ffn", 1, 2, 3, 4, 5, 6, 1, False, 7, 8, True)
    w = packed(ff)
    assert ff.linear_i4(1, w, out=2) == ("linear_i4", 1, w._constants, 2)
    assert w.dequantize(out=3) == ("dequantize_i4", w._constants, 3)
    assert w.shape == (8, 64) and w.group == 32 and "8 x 64" in repr(w)


def test_refusals_without_a_gpu(ff):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: ff.residual_norm(x, weight=x[0]), lambda: ff.residual_norm_backward(x, None, x, None, x[0]),
                 lambda: ff.moe_ffn(x, x, x, x, x, 1), lambda: ff.pack_i4(x.to(torch.uint8), x, group=32), lambda: ff.quantize_i4(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="kind"):
        ff.residual_norm(x, weight=x[0], kind="batch")
    with pytest.raises(TypeError, match="Int4Weight"):
        ff.linear_i4(x, x)
