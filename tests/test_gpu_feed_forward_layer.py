"""The operators together, as the example uses them: a tensor-parallel
feed-forward layer trained and served over virtual ranks, against the
unsharded layer in 64 bits."""
import importlib.util
import os

import pytest
import torch

from shot_allreduce_ranks_gb300 import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("ranks,tokens,hidden,width", [(4, 64, 512, 200), (2, 130, 264, 72), (8, 16, 1024, 136)])
def test_layer_over_ranks(ranks, tokens, hidden, width):
    build.build()
    spec = importlib.util.spec_from_file_location(
        "tensor_parallel_feed_forward", os.path.join(ROOT, "examples", "tensor_parallel_feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(ranks, tokens, hidden, width, say=lambda s: None)
    assert found["ranks agree"] and found["blocks agree"]
    # Each rounding to bfloat16 moves a value by at most u = 2^-8 of itself, so
    # its vector by at most u in norm.  Forward: h, the partial product, the sum and
    # y; a gradient passes at most eight (h, parts, ds, dh, gate and up, dgate or
    # dup, the product, the sum), and errors that a product of random weights
    # carries on keep their relative size.
    u = 2.0 ** -8
    assert found["y"] < 4 * u
    for k in ("dx", "dw_gate", "dw_up", "dw_down"):
        assert found[k] < 8 * u, k
    # 8 bits: steps of absmax / 127 with absmax below 6 standard deviations for
    # these sizes (h, a product of two normals' kind, below 16), errors uniform in a step: 16 / 127 /
    # sqrt(12) = 0.037 for h and 6 / 127 / sqrt(12) = 0.014 for the weights, added in squares.
    assert found["served"] < 4 * u + (0.037 ** 2 + 0.014 ** 2) ** 0.5
    torch.cuda.synchronize()


def test_no_wait_gave_up():
    from shot_allreduce_ranks_gb300 import _lib, ops_device_status
    assert ops_device_status() == _lib.AR_OK
