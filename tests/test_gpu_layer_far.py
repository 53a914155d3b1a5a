"""Rows and experts that lie further apart than 32 bits of elements."""
import pytest
import torch

from shot_allreduce_ranks_gb300 import build
from tests import layer_reference as layer
from tests.ff_reference import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


@pytest.fixture(scope="module")
def buffer():
    yield torch.zeros((1 << 32) + (1 << 24), dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("gap", [1 << 31, (1 << 31) + 3])
def test_rows_far_apart(ar, buffer, gap):
    g = torch.Generator(device=DEV).manual_seed(1)

    def far(at):
        t = buffer.as_strided((3, 1000), (gap, 1), at)
        t.copy_(torch.randn(3, 1000, generator=g, device=DEV))
        return t

    x, res, r, y = (far(at * 4096) for at in range(4))
    w, wa = (torch.randn(1000, generator=g, device=DEV).bfloat16() for _ in range(2))
    a = dict(weight=w, after_weight=wa)
    ar.residual_norm(x, res, r=r, y=y, **a)
    (want_r, er), (want_y, ey) = layer.Norm(x, res, **a).forward()
    assert_close(r, want_r, er, "r")
    assert_close(y, want_y, ey, "y")
    dy, dr = far(5 * 4096), far(6 * 4096)
    got = ar.residual_norm_backward(dy, dr, x, r, **a)
    want = layer.Norm(x, res, **a).backward(dy, dr, r)
    for t, name in zip(got, ("dx", "dresidual", "dweight")):
        assert_close(t, *want[name], name)
    # and a product whose rows of x and of the result do
    q = torch.randint(0, 16, (40, 1000), generator=g, device=DEV, dtype=torch.uint8)
    scale = torch.rand(40, 32, generator=g, device=DEV).bfloat16()
    out = buffer.as_strided((3, 40), (gap, 1), 7 * 4096)
    ar.linear_i4(x, ar.pack_i4(q, scale, group=32), out=out)
    wd = layer.weights_i4(q, scale, None, 32)
    assert_close(out, x.double() @ wd.T, 1004 * 2.0 ** -23 * (x.double().abs() @ wd.abs().T), "linear_i4")


def test_experts_far_apart(ar, buffer):
    g = torch.Generator(device=DEV).manual_seed(2)
    E, F, K = 3, 40, 136

    def far(at, rows, cols):
        t = buffer.as_strided((E, rows, cols), (1 << 31, cols, 1), at)
        t.copy_(torch.randn(E, rows, cols, generator=g, device=DEV) * cols ** -0.5)
        return t

    t = [torch.randn(5, K, generator=g, device=DEV).bfloat16(), torch.randn(5, E, generator=g, device=DEV), far(0, F, K), far(1 << 16, F, K),
         far(1 << 17, K, F)]
    want = layer.moe(*t, 2)
    assert_close(ar.moe_ffn(*t, 2), want[0], want[1], "moe_ffn")
