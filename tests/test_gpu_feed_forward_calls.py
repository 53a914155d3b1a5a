"""What the feed-forward operators do with values, handles and tensors at the edges of their contracts."""
import gc
import warnings

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


def normal(g, rows, cols, dtype=BF16, scale=1.0):
    return (torch.randn(rows, cols, generator=g, device=DEV) * scale).to(dtype)


def same_kind(got, want, unknown):
    """Infinities where the definition has them, with its sign, NaN where it has NaN, numbers elsewhere."""
    got = got.double()
    same = torch.where(torch.isfinite(want), torch.isfinite(got), (got == want) | (torch.isnan(got) & torch.isnan(want)))
    return bool((same | unknown).all())


@pytest.mark.parametrize("M", [3, 16, 40, 64, 65, 200])
@pytest.mark.parametrize("dtype,act", [(BF16, "silu"), (FP16, "gelu")])
@pytest.mark.parametrize("K,F", [(136, 72), (131, 77)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_gradients_of_operands_that_are_not_finite(ar, M, dtype, act, K, F, bad):
    """An infinity in x or in a weight makes the sums that it takes part in infinite, not NaN, at any number of
    tokens."""
    g = torch.Generator(device=DEV).manual_seed(M)
    x, wg, wu = normal(g, M, K, dtype), normal(g, F, K, dtype), normal(g, F, K, dtype)

    def away(t):  # no value below 1/8, where a product of three could vanish in 16 bits
        return torch.where(t.abs() < 0.125, torch.full_like(t, 0.125), t)

    gate, up, dout = (away(normal(g, M, F, dtype)) for _ in range(3))
    x[M - 1, 5] = bad
    wg[F - 2, 7] = bad
    wu[3, K - 1] = bad
    with ar.GatedFFN(M, K, F, dtype=dtype, activation=act, train=True) as ffn:
        dx, dwg, dwu = ffn.backward(x, wg, wu, gate, up, dout)
    f, df, _, edf = ref.activation(gate.double(), act)
    a, b = dout.double() * up.double() * df, dout.double() * f
    # where the slope's sign lies within its rounding, or a factor may be 0 in 16 bits, either is right
    near_a, near_b = (df.abs() <= edf) | (a.abs() <= 2 * ref.TINY[dtype]), b.abs() <= 2 * ref.TINY[dtype]
    # on the host: the definition's own infinities, summed one by one
    a, b, xd, wgd, wud = (t.double().cpu() for t in (a, b, x, wg, wu))
    near_a, near_b, bad_x, bad_g, bad_u = (t.double().cpu() for t in (near_a, near_b, *(~torch.isfinite(t) for t in (x, wg, wu))))
    for got, want, unknown, what in ((dx, a @ wgd + b @ wud, near_a @ bad_g + near_b @ bad_u, "dx"),
                                     (dwg, a.T @ xd, near_a.T @ bad_x, "dw_gate"), (dwu, b.T @ xd, near_b.T @ bad_x, "dw_up")):
        assert not torch.isfinite(want).all() and (unknown == 0).any()
        assert same_kind(got.cpu(), want, unknown > 0), what


@pytest.mark.parametrize("cols", [1, 2, 3, 5, 7, 9, 12, 15, 30, 33, 34, 67, 71, 100, 131, 257, 715])
@pytest.mark.parametrize("M", [20, 40, 150, 300])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_nothing_is_written_past_a_row(ar, cols, M, dtype):
    """Outputs are the first columns of a wider matrix whose rows start on 16 bytes; the others hold a marker."""
    g = torch.Generator(device=DEV).manual_seed(cols)
    ld = (cols + 15) // 8 * 8

    def wide(rows):
        buf = torch.full((rows + 2, ld), 7.0, dtype=dtype, device=DEV)
        return buf, buf[:rows, :cols]

    def untouched(buf, rows):
        return bool((buf[:rows, cols:] == 7).all()) and bool((buf[rows:] == 7).all())

    # the columns of a forward product's outputs are the shard's width
    x, wg, wu = normal(g, M, 72, dtype), normal(g, cols, 72, dtype, 0.1), normal(g, cols, 72, dtype, 0.1)
    bufs, outs = zip(*(wide(M) for _ in range(3)))
    with ar.GatedFFN(M, 72, cols, dtype=dtype) as ffn:
        got = ffn.forward(x, wg, wu, *outs)
    want, bounds = ref.forward(x, wg, wu, "silu")
    for a, b, e, what in zip(got, want, bounds, ("out", "gate", "up")):
        ref.assert_close(a, b, e, what)
    assert all(untouched(b, M) for b in bufs)

    # those of the gradients its hidden size
    F = 72
    x, wg, wu = normal(g, M, cols, dtype), normal(g, F, cols, dtype, 0.1), normal(g, F, cols, dtype, 0.1)
    gate, up, dout = (normal(g, M, F, dtype) for _ in range(3))
    bufs, outs = zip(*(wide(rows) for rows in (M, F, F)))
    with ar.GatedFFN(M, cols, F, dtype=dtype, train=True) as ffn:
        got = ffn.backward(x, wg, wu, gate, up, dout, *outs)
    want, bounds = ref.backward(x, wg, wu, gate, up, dout, "silu", two_parts=M <= 64)
    for a, b, e, what in zip(got, want, bounds, ("dx", "dw_gate", "dw_up")):
        ref.assert_close(a, b, e, what)
    assert all(untouched(b, rows) for b, rows in zip(bufs, (M, F, F)))

    # and those of an 8-bit product its channels
    q, w8 = (torch.randint(-127, 128, (n, 80), generator=g, device=DEV, dtype=torch.int8) for n in (M, cols))
    buf, out = wide(M)
    ar.linear_i8(q, torch.ones(M, device=DEV), w8, torch.ones(cols, device=DEV) / 4096, out=out)
    want = q.double() @ w8.double().T / 4096
    ref.assert_close(out, want, 0 * want, "linear_i8")
    assert untouched(buf, M)


def small(ar, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    M, K, F = 40, 64, 72
    return (M, K, F), (normal(g, M, K), normal(g, F, K), normal(g, F, K), *(normal(g, M, F) for _ in range(3)))


def test_a_handle_collected_while_a_graph_is_captured(ar):
    """Its workspace is freed later: freeing waits for the device, which would end the capture."""
    (M, K, F), t = small(ar)
    ffn = ar.GatedFFN(M, K, F, train=True)
    ffn.backward(*t)
    torch.cuda.synchronize()
    graph, x = torch.cuda.CUDAGraph(), torch.ones(8, device=DEV)
    with torch.cuda.graph(graph):
        y = x + 1
        del ffn
        gc.collect()
        z = y * 2
    graph.replay()
    torch.cuda.synchronize()
    assert bool((z == 4).all())


def test_a_handle_is_not_closed_while_a_graph_is_captured(ar):
    """Asked for by name, it is refused before the capture is broken."""
    (M, K, F), t = small(ar)
    ffn = ar.GatedFFN(M, K, F, train=True)
    graph, x = torch.cuda.CUDAGraph(), torch.ones(8, device=DEV)
    with torch.cuda.graph(graph):
        y = x + 1
        with pytest.raises(RuntimeError, match="captured"):
            ffn.close()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((y == 2).all())
    ffn.close()


def test_a_captured_backward_keeps_its_workspace(ar):
    """The graph holds the workspace's address, so dropping the handle does not free it."""
    (M, K, F), t = small(ar)
    ffn = ar.GatedFFN(M, K, F, train=True)
    want = ffn.backward(*t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ffn.backward(*t)
    assert ffn.captured
    del ffn
    gc.collect()
    others = [ar.GatedFFN(M, K, F, train=True) for _ in range(3)]
    for o in others:
        o.backward(*t[:5], t[5] * 3)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for o in others:
        assert not o.captured
        o.close()


def test_gradients_are_not_lost_without_a_word(ar):
    (M, K, F), (x, wg, wu, *_) = small(ar)
    p = torch.nn.Parameter(wg)
    w8, s8 = torch.ones(8, F, dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    with ar.GatedFFN(M, K, F) as ffn:
        with pytest.warns(UserWarning, match="w_gate requires grad"):
            h = ffn.forward(x, p, wu)
        assert not h.requires_grad
        with pytest.warns(UserWarning, match="x requires grad"):
            ar.dropout(x.clone().requires_grad_(), 0.5, 1)
        with pytest.warns(UserWarning, match="residual requires grad"):
            ar.dropout(x, 0.5, 1, residual=x.clone().requires_grad_())
        with pytest.warns(UserWarning, match="x requires grad"):
            q, s = ar.quantize_rows(h.clone().requires_grad_())
        with pytest.warns(UserWarning, match="w_scale requires grad"):
            ar.linear_i8(q, s, w8, s8.clone().requires_grad_())
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                ffn.forward(x, p, wu)
                ar.dropout(x.clone().requires_grad_(), 0.5, 1)
            ffn.forward(x, wg, wu)
            ar.linear_i8(q, s, w8, s8)
        with warnings.catch_warnings(), pytest.raises(UserWarning):
            warnings.simplefilter("error")
            ffn.forward(x, p, wu)
