"""Products with 4-bit weights, their layout and their quantisation, against the 64-bit definition."""
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


def weights(seed, N, K, group, zero, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    groups = -(-K // group)
    q = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=torch.uint8)
    scale = ((torch.rand((N, groups), generator=g, device=DEV) + 0.5) / 8).to(dtype)
    z = torch.randint(0, 16, (N, groups), generator=g, device=DEV, dtype=torch.uint8) if zero else None
    return q, scale, z


def tokens(seed, M, K, dtype, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 1000)
    return torch.randn((M, K + pad), generator=g, device=DEV).to(dtype)[:, :K]


def check(ar, x, q, scale, z, group, **k):
    y = ar.linear_i4(x, ar.pack_i4(q, scale, z, group=group), **k)
    w = layer.weights_i4(q, scale, z, group)
    # products are exact; a sum of K of them and the scaling of each group's part, in any order
    ff.assert_close(y, x.double() @ w.T, (x.shape[1] + 4) * ff.E32 * (x.double().abs() @ w.abs().T), "y")
    return y


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 65, 200])
@pytest.mark.parametrize("N,K", [(16, 64), (1, 1), (40, 128), (17, 130), (333, 200), (96, 2048), (50, 1091)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero,dtype", [(False, BF16), (True, BF16), (True, FP16), (False, FP16)])
def test_against_the_definition(ar, M, N, K, group, zero, dtype):
    check(ar, tokens(M, M, K, dtype), *weights(N + K, N, K, group, zero, dtype), group)


@pytest.mark.parametrize("N,K", [(8192, 512), (16, 16384), (1000, 5001), (5120, 1736), (64, 9000)])
@pytest.mark.parametrize("M", [1, 13, 40])
@pytest.mark.parametrize("group", [32, 128])
def test_larger(ar, N, K, M, group):
    check(ar, tokens(M, M, K, FP16), *weights(N + K, N, K, group, True, FP16), group)


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("M", [1, 5, 20])
def test_rows_of_wider_matrices(ar, pad, M):
    N, K = 70, 264
    q, scale, z = weights(1, N, K + pad, 32, True, BF16)
    buf = torch.full((M + 1, N + pad), 7.0, dtype=BF16, device=DEV)
    x = tokens(2, M, K, BF16, pad)
    y = check(ar, x, q[:, :K], scale[:, :-(-K // 32)], z[:, :-(-K // 32)], 32, out=buf[:M, :N])
    assert y.data_ptr() == buf.data_ptr()
    assert bool((buf[:M, N:] == 7).all()) and bool((buf[M:] == 7).all())
    # a row that begins at an odd place
    flat = tokens(3, 1, M * K + 1, BF16).reshape(-1)[1:].view(M, K)
    check(ar, flat, q[:, :K], scale[:, :-(-K // 32)], None, 32)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 64), (37, 300), (130, 1024)])
def test_quantisation(ar, dtype, zero, group, N, K):
    """Whole numbers, scales and zero points are those of the definition: the weights come back equal, and products with
    both are the same bits."""
    w = tokens(N, N, K, dtype, 3) * 0.1
    w[0, : min(K, 32)] = 0
    packed = ar.quantize_i4(w, group=group, zero=zero)
    assert packed.shape == (N, K) and packed.group == group and packed.dtype == dtype and (packed.zero is not None) == zero
    q, scale, z = layer.quantize_i4(w, group, zero)
    again = ar.pack_i4(q, scale, z, group=group)
    assert torch.equal(packed.data, again.data) and torch.equal(packed.scale, again.scale)
    assert not zero or torch.equal(packed.zero, again.zero)
    back = packed.dequantize()
    assert torch.equal(back, layer.weights_i4(q, scale, z, group).to(dtype))
    # half a step; with the zero point rounded and the ends cut one step more, and the roundings of scale and result
    step = scale.double().repeat_interleave(group, 1)[:, :K]
    assert bool(((back.double() - w.double()).abs() <= step * (1.51 if zero else 0.51) + 16 * ff.U[dtype] * step + ff.TINY[dtype]).all())
    x = tokens(1, 5, K, dtype)
    assert torch.equal(ar.linear_i4(x, packed), ar.linear_i4(x, again))


def test_quantisation_at_the_edges(ar):
    w = torch.zeros(6, 64, device=DEV, dtype=FP16)
    w[1, 3], w[2, 40], w[3] = float("inf"), float("nan"), 65504.0
    w[4, 0], w[4, 1] = 65504.0, -65504.0
    w[5] = 2.0 ** -24
    for zero in (False, True):
        packed = ar.quantize_i4(w, group=32, zero=zero)
        back = packed.dequantize()
        q, scale, z = layer.quantize_i4(w, 32, zero)
        assert torch.equal(torch.isnan(back), torch.isnan(layer.weights_i4(q, scale, z, 32)))
        fine = torch.isfinite(back)
        assert torch.equal(back[fine], layer.weights_i4(q, scale, z, 32).to(FP16)[fine])
        assert bool(torch.isnan(back[1, :32]).all()) and bool((back[1, 32:] == 0).all()) and bool((back[0] == 0).all())
        y = ar.linear_i4(torch.ones(1, 64, device=DEV, dtype=FP16), packed)
        assert torch.isnan(y[0, 1]) and torch.isnan(y[0, 2]) and y[0, 0] == 0


def test_values_that_are_not_finite(ar):
    """An infinity in x or in a scale reaches its own results alone, as the definition has it."""
    M, N, K, group = 12, 40, 500, 128
    x, (q, scale, z) = tokens(1, M, K, BF16), weights(5, N, K, group, True, BF16)
    want = check(ar, x, q, scale, z, group)
    scale2 = scale.clone()
    scale2[7, 3] = float("inf")
    got = ar.linear_i4(x, ar.pack_i4(q, scale2, z, group=group))
    others = torch.arange(N, device=DEV) != 7
    assert torch.equal(got[:, others], want[:, others])
    part = x[:, 384:].double() @ (q[7, 384:].double() - z[7, 3].double())
    assert torch.equal(got[:, 7].double(), part * float("inf"))
    x2 = x.clone()
    x2[3, 9] = float("inf")
    got = ar.linear_i4(x2, ar.pack_i4(q, scale, z, group=group))
    rows = torch.arange(M, device=DEV) != 3
    assert torch.equal(got[rows], want[rows]) and not bool(torch.isfinite(got[3]).any())


def test_only_the_low_bits_count(ar):
    q, scale, z = weights(5, 20, 96, 32, True, BF16)
    a, b = ar.pack_i4(q, scale, z, group=32), ar.pack_i4(q | 0xF0, scale, z | 0xF0, group=32)
    assert torch.equal(a.data, b.data) and torch.equal(a.zero, b.zero)


def test_no_tokens(ar):
    w = ar.pack_i4(*weights(1, 24, 64, 64, False, BF16), group=64)
    assert ar.linear_i4(torch.empty(0, 64, dtype=BF16, device=DEV), w).shape == (0, 24)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (13, 333, 5001), (40, 2000, 2048)])
def test_the_same_bits_every_time_in_graphs_and_on_streams(ar, M, N, K):
    x, w = tokens(1, M, K, BF16), ar.pack_i4(*weights(2, N, K, 64, True, BF16), group=64)
    want = ar.linear_i4(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = ar.linear_i4(x, w, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ar.linear_i4(x, w)
    for _ in range(20):
        graph.replay()
        assert torch.equal(out, want) and torch.equal(ar.linear_i4(x, w), want)
    x.copy_(x.flip(1))
    graph.replay()
    assert torch.equal(out, ar.linear_i4(x, w)) and not torch.equal(out, want)


def test_refusals(ar):
    q, scale, z = weights(1, 24, 96, 32, True, BF16)
    w, x = ar.pack_i4(q, scale, z, group=32), tokens(1, 3, 96, BF16)
    for call, what in ((lambda: ar.pack_i4(q, scale, z, group=48), "group must be"), (lambda: ar.pack_i4(q.int(), scale, group=32), "q must be"),
                       (lambda: ar.pack_i4(q, scale[:, :2], group=32), "scale must be 24 x 3"), (lambda: ar.pack_i4(q, scale, z[:20], group=32), "zero must be 24"),
                       (lambda: ar.pack_i4(q, scale.float(), group=32), "scale must be torch.bfloat16 or"), (lambda: ar.pack_i4(q[:0], scale[:0], group=32), "1 to 2"),
                       (lambda: ar.quantize_i4(x.float()), "w must be"), (lambda: ar.quantize_i4(x, group=16), "group must be"),
                       (lambda: ar.linear_i4(x[:, :95], w), "x must be . x 96"), (lambda: ar.linear_i4(x.half(), w), "x must be a 2-D torch.bfloat16"),
                       (lambda: ar.linear_i4(x, w, out=x), "out must be 3 x 24"), (lambda: ar.linear_i4(x.T, w), "x must be . x 96"),
                       (lambda: ar.linear_i4(x, ar.Int4Weight(w.data[:-16], w.scale, w.zero, (24, 96), 32)), "weight's data must be"),
                       (lambda: ar.linear_i4(x, ar.Int4Weight(w.data, w.scale, w.zero[1:], (24, 96), 32)), "weight's zero must be"),
                       (lambda: ar.linear_i4(x, ar.Int4Weight(w.data, w.scale, w.zero, (24, 96), 64)), "weight's")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError, match="Int4Weight"):
        ar.linear_i4(x, q)
    with pytest.warns(UserWarning, match="x requires grad"):
        ar.linear_i4(x.clone().requires_grad_(), w)
