"""What is between the experts' two products reaches the second in two parts, so that its rounding does not show in the
result: bounds with the square of a half step where one 16-bit number would leave a whole one."""
import pytest
import torch

from shot_allreduce_ranks_gb300 import build
from tests import ff_reference as ff
from tests import layer_reference as layer

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def inputs(seed, T, K, F, E, dtype, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    return [normal(T, K), normal(T, E, scale=1.5), normal(E, F, K, scale=gain * K ** -0.5), normal(E, F, K, scale=K ** -0.5),
            normal(E, K, F, scale=F ** -0.5)]


def definition(x, logits, w_gate, w_up, w_down, top_k, activation, normalize):
    """(out, its bound before the final rounding): that of layer_reference.moe, but for h as the sum of two numbers of the
    type.  The second is what the first's rounding left, at most u |h|, and is rounded itself: u^2 |h|, or half the type's
    smallest subnormal.  The second product doubles the number of products that are summed."""
    u, tiny = ff.U[x.dtype], ff.TINY[x.dtype]
    expert, weight, rel = layer.routing(logits, top_k, normalize)
    K, F = x.shape[1], w_gate.shape[1]
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    bound, size = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(w_gate.shape[0]):
        t, j = torch.nonzero(expert == e, as_tuple=True)
        if not len(t):
            continue
        w, ew = weight[t, j].to(x.device)[:, None], (weight[t, j] * rel[t, 0]).to(x.device)[:, None]
        t = t.to(x.device)
        (h, _, _), (eh, _, _) = ff.forward(x[t], w_gate[e], w_up[e], activation)
        eh = eh + u * u * (h.abs() + eh) + tiny
        d = w_down[e].double()
        part, epart = h @ d.T, (eh + 2 * F * ff.E32 * (h.abs() + eh)) @ d.abs().T
        out[t] += w * part
        bound[t] += w * epart + ew * (part.abs() + epart)
        size[t] += w * (part.abs() + epart)
    return out, bound + (top_k * (F / 64 + 1) + 10) * layer.E * size


# blocks of 8, 16 and 32 tokens an expert, more than one run of tokens, odd widths, pieces that end early
@pytest.mark.parametrize("T,K,F,E,top_k", [(1, 256, 1024, 4, 2), (9, 136, 72, 3, 1), (16, 520, 200, 2, 2), (32, 64, 264, 2, 2),
                                           (70, 131, 77, 3, 2), (20, 2048, 1031, 6, 3), (3, 40, 1, 2, 1)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act,normalize", [("silu", True), ("gelu", False)])
def test_the_rounding_between_the_products_does_not_show(ar, T, K, F, E, top_k, dtype, act, normalize):
    t = inputs(T + F, T, K, F, E, dtype)
    got = ar.moe_ffn(*t, top_k, activation=act, normalize=normalize)
    ff.assert_close(got, *definition(*t, top_k, act, normalize), "out")


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_infinities_between_the_products_stay_infinities(ar, dtype):
    """An h that is infinite has nothing left for its second part: its results are infinities and no NaN."""
    T, K, F = 5, 64, 40
    t = inputs(1, T, K, F, 1, dtype)
    t[0].fill_(1.0)
    t[2][0, 7].fill_(1.0)      # gate 64, act(64) = 64
    t[3][0, 7].fill_(float("inf"))  # h of inner row 7 is infinite
    t[4].abs_().clamp_(min=0.01)
    got = ar.moe_ffn(*t, 1)
    assert bool((got == float("inf")).all())


def test_the_smaller_workspace_of_the_c_call(ar):
    """With ar_moe_scratch_bytes of scratch h is one number; with ar_moe_two_part_scratch_bytes the call gives what the
    Python call gives, and what it leaves of the scratch behind that size is as it was."""
    import ctypes

    from shot_allreduce_ranks_gb300 import _lib
    lib = _lib.load()
    T, K, F, E = 12, 128, 200, 4
    x, z, wg, wu, wd = t = inputs(2, T, K, F, E, BF16)
    m = _lib.ArMoe(0, 0, 0, E, 0, E, 2, 1, K, F)
    small, two = lib.ar_moe_scratch_bytes(ctypes.byref(m), T), lib.ar_moe_two_part_scratch_bytes(ctypes.byref(m), T)
    results = []
    for n in (small, two - 1, two):
        room = torch.full((n + 64,), 77, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(x)
        assert lib.ar_moe_ffn(ctypes.byref(m), x.data_ptr(), K, z.data_ptr(), E, wg.data_ptr(), wu.data_ptr(), K, F * K, wd.data_ptr(), F,
                              K * F, out.data_ptr(), K, None, None, T, room.data_ptr(), n,
                              torch.cuda.current_stream().cuda_stream) == 0
        assert bool((room[n:] == 77).all())
        results.append(out)
    want = layer.moe(*t, 2)
    ff.assert_close(results[0], want[0], want[1], "one part")
    assert torch.equal(results[0], results[1])
    assert torch.equal(results[2], ar.moe_ffn(*t, 2)) and not torch.equal(results[2], results[0])
