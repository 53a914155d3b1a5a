"""The layer of gated experts for a few tokens against the 64-bit definition."""
import pytest
import torch

from shot_allreduce_ranks_gb300 import build
from tests import layer_reference as layer
from tests.ff_reference import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def inputs(seed, T, K, F, E, local=None, dtype=BF16, logits=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    local = E if local is None else local

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(to)

    return [normal(T, K), normal(T, E, scale=1.5, to=logits or dtype), normal(local, F, K, scale=K ** -0.5),
            normal(local, F, K, scale=K ** -0.5), normal(local, K, F, scale=F ** -0.5)]


def check(ar, t, top_k, **k):
    out, expert, weight = ar.moe_ffn(*t, top_k, routing=True, **k)
    want = layer.moe(*t, top_k, **k)
    assert torch.equal(expert.cpu(), want[2])
    off = (weight.double().cpu() - want[3]).abs()
    assert bool((off <= want[4] + 1e-37).all()), float(off.max())
    assert_close(out, want[0], want[1], "out")
    assert torch.equal(ar.moe_ffn(*t, top_k, **k), out)
    return out, expert, weight


# tokens, hidden, width, experts: one of each kernel's blocks of eight tokens, strips and pieces that end early, odd rows
@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 31, 32, 33, 70])
@pytest.mark.parametrize("K,F,E,top_k", [(64, 64, 4, 2), (136, 72, 8, 1), (2048, 256, 3, 3), (131, 77, 5, 2), (1, 1, 2, 1),
                                         (520, 1040, 16, 8), (40, 9, 300, 6), (24, 16, 70, 16)])
@pytest.mark.parametrize("dtype,act,normalize", [(BF16, "silu", True), (FP16, "gelu", False)])
def test_against_the_definition(ar, T, K, F, E, top_k, dtype, act, normalize):
    check(ar, inputs(T + K, T, K, F, E, dtype=dtype), top_k, activation=act, normalize=normalize)


@pytest.mark.parametrize("logits", [BF16, FP16, FP32])
@pytest.mark.parametrize("E", [1, 31, 64, 65, 256, 257, 1024])
def test_routing(ar, logits, E):
    """Every form of the search, with equal logits among them."""
    t = inputs(E, 32, 16, 8, E, dtype=FP16, logits=logits)
    t[1] = (t[1] * 2).round() / 2 if E > 1 else t[1]
    for top_k in {1, min(E, 5), min(E, 16)}:
        for normalize in (True, False):
            check(ar, t, top_k, normalize=normalize)


@pytest.mark.parametrize("first,local", [(0, 3), (5, 6), (10, 6), (15, 1)])
def test_a_part_of_the_experts(ar, first, local):
    """The parts' outputs sum to the whole layer's; a token whose experts are all elsewhere gets zeros."""
    t = inputs(first, 20, 96, 40, 16, local)
    out, expert, _ = check(ar, t, 2, first_expert=first)
    none = ((expert < first) | (expert >= first + local)).all(1)
    assert bool(none.any()) and bool((out[none] == 0).all()) and bool((out[~none] != 0).any())


@pytest.mark.parametrize("pad", [1, 4, 8])
@pytest.mark.parametrize("K,F", [(64, 48), (35, 21)])
def test_strides(ar, pad, K, F):
    """Gate and up projections as halves of one tensor, rows and experts further apart; nothing behind out is written."""
    T, E = 11, 6
    x, logits, *_ = inputs(pad, T, K, F, E)
    x = inputs(pad, T, K + pad, F, E)[0][:, :K]
    logits = torch.cat([logits, logits], 1)[:, :E]
    both = inputs(7, 1, K + pad, 2 * F + 1, E)[2][:, :, :K]
    down = inputs(8, 1, F + pad, K + 1, E)[2][:, :K, :F]
    buf = torch.full((T + 1, K + pad), 7.0, dtype=BF16, device=DEV)
    t = [x, logits, both[:, :F], both[:, F:2 * F], down]
    want = check(ar, t, 3)[0]
    got = ar.moe_ffn(*t, 3, out=buf[:T, :K])
    assert got.data_ptr() == buf.data_ptr() and torch.equal(got, want)
    assert bool((buf[:T, K:] == 7).all()) and bool((buf[T:] == 7).all())


def test_every_expert_the_same_matrix(ar):
    t = inputs(3, 9, 64, 32, 1)
    t[1] = inputs(3, 9, 64, 32, 12)[1]
    t[2:] = [w.expand(12, -1, -1) for w in t[2:]]
    check(ar, t, 4)


def test_all_tokens_to_one_expert(ar):
    t = inputs(4, 32, 256, 64, 8)
    t[1][:, 5] = 30.0
    check(ar, t, 1)
    check(ar, t, 3, normalize=False)


@pytest.mark.parametrize("E", [6, 100, 400])
def test_logits_at_the_edges(ar, E):
    inf, nan = float("inf"), float("nan")
    t = inputs(5, 9, 32, 24, E, logits=FP32)
    z = t[1]
    z[1] = -inf                      # nothing is left
    z[2, 1:] = -inf                  # one is left
    z[3] = 0.0                       # all equal
    z[3, 1::2] = -0.0
    z[4] = torch.finfo(FP32).min     # equal, the lowest value
    z[5, 2] = torch.finfo(FP32).max
    for normalize in (True, False):
        out, expert, weight = check(ar, t, 4, normalize=normalize)
        assert expert[1].tolist() == [-1] * 4 and bool((out[1] == 0).all()) and bool((weight[1] == 0).all())
        assert expert[2].tolist() == [0, -1, -1, -1] and weight[2].tolist() == [1, 0, 0, 0]
        assert expert[3].tolist() == expert[4].tolist() == [0, 1, 2, 3]
        assert expert[5, 0] == 2 and weight[5, 0] == 1
        bad = z.clone()
        bad[7, 3], bad[8, 4] = nan, inf
        o, e, w = ar.moe_ffn(t[0], bad, *t[2:], 4, normalize=normalize, routing=True)
        assert e[7, 0] == 3 and e[8, 0] == 4
        assert bool(torch.isnan(w[7:]).all()) and bool(torch.isnan(o[7:]).all())
        assert torch.equal(o[:7], out[:7]) and torch.equal(w[:7], weight[:7])


@pytest.mark.parametrize("T", [5, 30])
def test_values_that_are_not_finite_stay_with_their_tokens(ar, T):
    """An infinity in an expert's matrices reaches the tokens that were sent to it and no others."""
    t = inputs(6, T, 64, 40, 8)
    want, expert, _ = check(ar, t, 2)
    t[2][3, 5, 7] = float("inf")
    t[4][3, 9, 2] = float("inf")
    got = ar.moe_ffn(*t, 2)
    sent = (expert == 3).any(1)
    assert bool(sent.any()) and not bool(sent.all())
    assert torch.equal(got[~sent], want[~sent])
    assert not bool(torch.isfinite(got[sent]).all())
    t = inputs(6, T, 64, 40, 8)
    t[0][2, 9] = float("nan")
    got = ar.moe_ffn(*t, 2)
    others = torch.arange(T, device=DEV) != 2
    assert torch.equal(got[others], want[others]) and bool(torch.isnan(got[2]).all())


def test_no_tokens(ar):
    t = inputs(7, 0, 32, 16, 4)
    out, expert, weight = ar.moe_ffn(*t, 2, routing=True)
    assert out.shape == (0, 32) and expert.shape == weight.shape == (0, 2)


@pytest.mark.parametrize("T,K,F,E,k", [(1, 2048, 512, 16, 4), (32, 1024, 264, 64, 8), (45, 136, 72, 8, 2)])
def test_the_same_bits_every_time_in_graphs_and_on_streams(ar, T, K, F, E, k):
    t = inputs(9, T, K, F, E)
    want = ar.moe_ffn(*t, k, routing=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ar.moe_ffn(*t, k, routing=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ar.moe_ffn(*t, k, routing=True)
        graphs.append((g, out, torch.cuda.Stream()))
    for _ in range(20):
        for g, _, s in graphs:  # side by side: each has scratch memory of its own
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out, _ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(ar.moe_ffn(*t, k, routing=True), want))
    # other values in the same places
    t[1].copy_(t[1].flip(1))
    t[0].copy_(t[0].flip(0))
    graphs[0][0].replay()
    again = ar.moe_ffn(*t, k, routing=True)
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], again)) and not torch.equal(again[0], want[0])


def test_refusals(ar):
    t = inputs(10, 4, 32, 16, 6)
    x, z, wg, wu, wd = t
    for args, what in (((x.float(), z, wg, wu, wd, 2), "x must be torch.bfloat16"), ((x, z[:3], wg, wu, wd, 2), "logits must be 4"),
                       ((x, z.to(torch.int32), wg, wu, wd, 2), "logits must be"), ((x, z, wg[:, :, :31], wu, wd, 2), "w_gate has size 31"),
                       ((x, z, wg, wu[:5], wd, 2), "w_up has size 5"), ((x, z, wg, wu, wd[:, :, :9], 2), "w_down has size 9"),
                       ((x, z, wg, wu.half(), wd, 2), "w_up must be a 3-D"), ((x, z, wg[0], wu, wd, 2), "w_gate must be a 3-D"),
                       ((x, z, wg, wu.repeat(1, 2, 1)[:, :16], wd, 2), "same strides"), ((x, z, wg, wu, wd, 0), "top_k"),
                       ((x, z, wg, wu, wd, 7), "top_k"), ((x, z[:, :5], wg, wu, wd, 2), "not among the 5"),
                       ((x, z, wg.mT.contiguous().mT, wu, wd, 2), "contiguous rows")):
        with pytest.raises(ValueError, match=what):
            ar.moe_ffn(*args)
    with pytest.raises(ValueError, match="not among the 6"):
        ar.moe_ffn(*t, 2, first_expert=1)
    with pytest.raises(ValueError, match="activation"):
        ar.moe_ffn(*t, 2, activation="relu")
    with pytest.warns(UserWarning, match="w_up requires grad"):
        ar.moe_ffn(x, z, wg, wu.clone().requires_grad_(), wd, 2)
