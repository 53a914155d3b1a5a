"""Products whose tiles lie partly past the last row, hundreds of times.

A warp of the tensor-core kernel stores a tile through two boxes in shared
memory that take turns.  In the sizes below a CTA makes several tiles, some
warps' rows of a tile lie past the last one, and contractions are short, so
that the next tile's values are ready while the copy engine still reads the
last one's boxes.  Outputs hold a marker before every call; the first call is
held to the 64-bit formula and the others to its bits.
"""
import pytest
import torch

from shot_allreduce_ranks_gb300 import build
from tests import ff_reference as ref

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
DEV = "cuda"


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def inputs(M, K, F, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(rows, cols, scale=1.0):
        return (torch.randn(rows, cols, generator=g, device=DEV) * scale).to(dtype)

    return normal(M, K), normal(F, K, K ** -0.5), normal(F, K, K ** -0.5), [normal(M, F) for _ in range(3)]


def repeat(call, outs, times):
    """The outputs of the first call; how many values of the later ones differ from it, or keep the marker."""
    def run():
        for t in outs:
            t.fill_(float("nan"))
        call()

    run()
    first = [t.clone() for t in outs]
    off = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(times):
        run()
        for t, f in zip(outs, first):
            off += (t != f).sum()  # a NaN differs too
    return first, int(off)


@pytest.mark.parametrize("M,K,F,dtype,act", [
    (600, 128, 3584, BF16, "silu"), (1030, 64, 1736, FP16, "gelu"), (1500, 72, 8192, BF16, "gelu"), (2100, 256, 3584, FP16, "silu")])
@pytest.mark.parametrize("save", [True, False])
def test_forward(ar, M, K, F, dtype, act, save):
    x, wg, wu, _ = inputs(M, K, F, dtype, M)
    outs = [torch.empty(M, F, dtype=dtype, device=DEV) for _ in range(3 if save else 1)]
    with ar.GatedFFN(M, K, F, dtype=dtype, activation=act) as ffn:
        first, off = repeat(lambda: ffn.forward(x, wg, wu, *outs), outs, 300)
    want, bounds = ref.forward(x, wg, wu, act)
    for a, b, e, what in zip(first, want, bounds, ("out", "gate", "up")):
        ref.assert_close(a, b, e, what)
    assert off == 0


@pytest.mark.parametrize("M,K,F,dtype,act", [
    (440, 5120, 1736, BF16, "silu"), (200, 5120, 3400, BF16, "gelu"), (80, 512, 3400, FP16, "silu"),
    # up to 64 tokens: two parts of each value, blocks of 16 tokens
    (40, 5120, 1736, FP16, "gelu"), (64, 8192, 1304, BF16, "silu"), (20, 8192, 3400, FP16, "silu")])
def test_gradients(ar, M, K, F, dtype, act):
    x, wg, wu, (gate, up, dout) = inputs(M, K, F, dtype, M)
    outs = [torch.empty(*s, dtype=dtype, device=DEV) for s in ((M, K), (F, K), (F, K))]
    with ar.GatedFFN(M, K, F, dtype=dtype, activation=act, train=True) as ffn:
        first, off = repeat(lambda: ffn.backward(x, wg, wu, gate, up, dout, *outs), outs, 200)
    want, bounds = ref.backward(x, wg, wu, gate, up, dout, act, two_parts=M <= 64)
    for a, b, e, what in zip(first, want, bounds, ("dx", "dw_gate", "dw_up")):
        ref.assert_close(a, b, e, what)
    assert off == 0


def test_no_wait_gave_up(ar):
    assert ar.ops_device_status() == 0
