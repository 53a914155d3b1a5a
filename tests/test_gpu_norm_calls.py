"""Calls of the norms that their documentation allows, or that are refused."""
import pytest
import torch

from shot_allreduce_ranks_gb300 import build

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF16)


def off_16(t):
    """The same values, one element off a multiple of 16 bytes."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    flat[1:].copy_(t.reshape(-1))
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("rows,cols", [(40, 16384), (300, 1024)])
def test_arrays_that_are_not_read_change_nothing(ar, rows, cols):
    """Without gate and after_weight x is not read, without weight r is not, without a gate after_bias is not: where they lie does not change a bit."""
    dy, dr, x, r, w = normal(1, rows, cols), normal(2, rows, cols), normal(3, rows, cols), normal(4, rows, cols), normal(5, cols)
    want = ar.residual_norm_backward(dy, dr, None, r, w)
    for other in (x, off_16(x)):
        got = ar.residual_norm_backward(dy, dr, other, r, w)
        assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)
    want = ar.residual_norm_backward(None, dr, x, None, None, None, w)
    for other in (r, off_16(r)):
        got = ar.residual_norm_backward(None, dr, x, other, None, None, w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[4], want[4])
    b = normal(6, cols)
    want = ar.residual_norm_backward(None, dr, x, None, None, None, w, b)
    got = ar.residual_norm_backward(None, dr, x, None, None, None, w, off_16(b))
    assert all(torch.equal(got[i], want[i]) for i in (0, 4, 5))


def test_r_and_y_are_two_tensors(ar):
    x, res, w = normal(1, 6, 40), normal(2, 6, 40), normal(3, 40)
    keep = x.clone()
    with pytest.raises(ValueError, match="r and y"):
        ar.residual_norm(x, res, w, r=x, y=x)
    assert torch.equal(x, keep)
    both = torch.empty(6, 80, dtype=BF16, device=DEV)
    r, y = ar.residual_norm(x, res, w, r=both[:, :40], y=both[:, 40:])
    want = ar.residual_norm(x, res, w)
    assert torch.equal(r, want[0]) and torch.equal(y, want[1])
