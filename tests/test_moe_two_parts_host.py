"""The larger workspace of the layer of experts; no GPU is touched."""
import ctypes

import pytest

from shot_allreduce_ranks_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_the_second_part_is_as_large_as_the_first(lib):
    def both(tokens, **k):
        d = dict(dtype=0, logits_dtype=2, activation=0, experts=8, first_expert=2, local_experts=4, top_k=3, normalize=1, hidden=16, width=12)
        m = _lib.ArMoe(*dict(d, **k).values())
        return [f(ctypes.byref(m), tokens) for f in (lib.ar_moe_scratch_bytes, lib.ar_moe_two_part_scratch_bytes)]

    # a row of 16-bit numbers for each choice of each token, whole groups of eight
    for tokens, width in ((5, 12), (1, 17), (31, 1000), (32, 8), (1000, 8)):
        one, two = both(tokens, width=width)
        assert two - one == min(tokens, 32) * 3 * -(-width // 8) * 8 * 2 and two % 16 == 0
    assert both(0) == [0, 0] and both(5, top_k=9) == [0, 0] and lib.ar_moe_two_part_scratch_bytes(None, 5) == 0
