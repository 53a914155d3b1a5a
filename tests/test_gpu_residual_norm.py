"""Norms with the gate and the residual, forward and backward, against the 64-bit formulas."""
import pytest
import torch

from shot_allreduce_ranks_gb300 import build
from tests import layer_reference as layer
from tests.ff_reference import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("dx", "dresidual", "dweight", "dbias", "dafter_weight", "dafter_bias", "dgate")

# (rows, cols): one element, less than a group, odd rows, a row a warp, several warps, wide ones, past what stays in registers
SIZES = [(1, 1), (3, 7), (2, 64), (65, 136), (33, 1031), (1, 5120), (440, 520), (9, 4104), (5, 8192), (3, 16384), (2, 20007)]
# what is there: the residual, the norm after the block, the norm before the next, biases, gate rows (-1: one a row)
PARTS = [dict(), dict(residual=True), dict(residual=True, after=True, scale=0.7, offset=1.0),
         dict(residual=True, after=True, before=False, bias=True), dict(residual=True, bias=True, gates=-1),
         dict(residual=True, after=True, bias=True, gates=1, scale=-1.5), dict(after=True, gates=1, offset=1.0)]


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def inputs(seed, rows, cols, dtype, residual=False, after=False, before=True, bias=False, gates=0, scale=1.0, offset=0.0,
           kind="rms", pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, mean=0.0, size=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * size + mean).to(dtype)

    def matrix(**k):
        return normal(rows, cols + pad, **k)[:, :cols]

    a = dict(kind=kind, eps=1e-5, residual_scale=scale, weight_offset=offset)
    x = matrix(mean=0.3)
    if residual:
        a["residual"] = matrix(size=2.0)
    if before:
        a["weight"] = normal(cols, mean=1.0 - offset, size=0.3)
        if bias:
            a["bias"] = normal(cols)
    if after:
        a["after_weight"] = normal(cols, mean=1.0 - offset, size=0.3)
        if bias:
            a["after_bias"] = normal(cols)
    if gates:
        a["gate"] = normal(rows if gates < 0 else gates, cols)
    return x, a, matrix


def check_forward(ar, x, a, **more):
    r, y = ar.residual_norm(x, **a, **more)
    want_r, want_y = layer.Norm(x, **a).forward()
    if r is not None:
        assert_close(r, *want_r, "r")
    else:
        assert not any(k in a for k in ("residual", "gate", "after_weight"))
    assert (y is None) == (want_y is None)
    if y is not None:
        assert_close(y, *want_y, "y")
    return r, y


def check_backward(ar, x, a, dy, dr, r):
    stored = r if r is not None else x
    back = {k: v for k, v in a.items() if k != "residual"}
    got = dict(zip(NAMES, ar.residual_norm_backward(dy, dr, x, r, **back)))
    want = layer.Norm(x, **a).backward(dy, dr, stored)
    if r is None:
        del want["dresidual"]
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k, v in want.items():
        assert_close(got[k], *v, k)
    return got


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward_and_backward(ar, rows, cols, parts, kind, dtype):
    x, a, matrix = inputs(rows + cols, rows, cols, dtype, kind=kind, **parts)
    r, _ = check_forward(ar, x, a)
    # Without a residual the stored r is the rounded one all the same.
    check_backward(ar, x, a, matrix() if "weight" in a else None, matrix() if r is not None else None, r)


@pytest.mark.parametrize("rows,gates", [(12, 3), (300, 100), (701, 701), (1500, 500), (1001, 7), (320, 320), (640, 2)])
@pytest.mark.parametrize("cols", [72, 333])
def test_gates_of_runs_of_rows(ar, rows, gates, cols):
    x, a, matrix = inputs(gates, rows, cols, BF16, residual=True, after=True, gates=gates)
    r, _ = check_forward(ar, x, a)
    check_backward(ar, x, a, matrix(), matrix(), r)


@pytest.mark.parametrize("pad", [1, 5, 8, 40])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [33, 256, 2056])
def test_rows_of_wider_matrices(ar, pad, dtype, cols):
    """Every operand has a row stride of its own; what lies behind the outputs' rows stays as it was."""
    rows = 19
    x, a, matrix = inputs(pad, rows, cols, dtype, residual=True, after=True, bias=True, gates=1, kind="layer", pad=pad)
    a["residual"] = torch.cat([a["residual"], a["residual"][:, :1]], 1)[:, :cols]
    outs = [torch.full((rows + 1, cols + extra), 7.0, dtype=dtype, device=DEV) for extra in (pad, 8)]
    views = [t[:rows, :cols] for t in outs]
    r, y = check_forward(ar, x, a, r=views[0], y=views[1])
    assert r.data_ptr() == views[0].data_ptr() and y.data_ptr() == views[1].data_ptr()
    assert all(bool((t[:rows, cols:] == 7).all()) and bool((t[rows:] == 7).all()) for t in outs)
    check_backward(ar, x, a, matrix(), matrix()[:, :], r)


@pytest.mark.parametrize("cols", [130, 5120, 20008])
def test_outputs_in_the_place_of_inputs(ar, cols):
    for swap in (False, True):
        x, a, _ = inputs(3, 21, cols, BF16, residual=True, after=True)
        want = ar.residual_norm(x, **a)
        keep = x.clone(), a["residual"].clone()
        to = (keep[1], keep[0]) if not swap else keep
        r, y = ar.residual_norm(keep[0], **dict(a, residual=keep[1]), r=to[0], y=to[1])
        assert torch.equal(r, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("cols", [100, 4096])
def test_a_mean_far_from_zero(ar, cols):
    """The variance is that of the differences from the mean, which squares of 1000 would bury."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(8, cols, generator=g, device=DEV) + 1000.0
    w = torch.ones(cols, device=DEV)
    check_forward(ar, x, dict(weight=w, kind="layer", eps=1e-5))
    check_backward(ar, x, dict(weight=w, kind="layer", eps=1e-5), torch.randn(8, cols, generator=g, device=DEV), None, None)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("cols", [65, 3000])
def test_values_that_are_not_finite_stay_in_their_row(ar, bad, kind, cols):
    x, a, matrix = inputs(5, 6, cols, BF16, residual=True, kind=kind)
    want = ar.residual_norm(x, **a)
    x2 = x.clone()
    x2[3, 7] = bad
    r, y = ar.residual_norm(x2, **a)
    others = [0, 1, 2, 4, 5]
    assert torch.equal(r[others], want[0][others]) and torch.equal(y[others], want[1][others])
    assert not torch.isfinite(r[3, 7]) and not torch.isfinite(y[3, 7])
    dy, dr = matrix(), matrix()
    back = {k: v for k, v in a.items() if k != "residual"}
    one = ar.residual_norm_backward(dy, dr, x, want[0], **back)
    two = ar.residual_norm_backward(dy, dr, x2, r, **back)
    assert torch.equal(one[0][others], two[0][others])


def test_rows_of_zeros(ar):
    x = torch.zeros(3, 40, dtype=BF16, device=DEV)
    w, b = torch.ones(40, dtype=BF16, device=DEV), torch.full((40,), 2.0, dtype=BF16, device=DEV)
    for kind in ("rms", "layer"):
        y = ar.residual_norm(x, weight=w, bias=b, kind=kind)[1]
        assert bool((y == 2).all())
        dx = ar.residual_norm_backward(torch.ones_like(x), None, x, None, w, b, kind=kind)[0]
        assert bool(torch.isfinite(dx).all())


def test_no_rows(ar):
    x, w = torch.empty(0, 24, dtype=BF16, device=DEV), torch.ones(24, dtype=BF16, device=DEV)
    r, y = ar.residual_norm(x, x, w, w)
    assert r.shape == y.shape == (0, 24)
    got = ar.residual_norm_backward(x, x, x, x, w, w)
    assert got[0].shape == (0, 24) and bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_gradients_that_are_one(ar):
    """Where nothing stands between x and the residual their gradients are one tensor; a scale or a gate parts them."""
    x, a, matrix = inputs(7, 5, 64, BF16, residual=True)
    r = ar.residual_norm(x, **a)[0]
    w = a["weight"]
    dx, dres, *_ = ar.residual_norm_backward(matrix(), matrix(), None, r, w)
    assert dx.data_ptr() == dres.data_ptr()
    dx, dres, *_ = ar.residual_norm_backward(matrix(), matrix(), None, r, w, residual_scale=0.5)
    assert dx.data_ptr() != dres.data_ptr() and torch.equal(dres, (dx.float() * 0.5).bfloat16())
    assert ar.residual_norm_backward(matrix(), matrix(), None, r, w, need_dresidual=False)[1] is None


@pytest.mark.parametrize("rows,cols", [(440, 5120), (701, 333)])
def test_the_same_bits_every_time_and_in_a_graph(ar, rows, cols):
    x, a, matrix = inputs(11, rows, cols, BF16, residual=True, after=True, bias=True, gates=1, kind="layer")
    back = {k: v for k, v in a.items() if k != "residual"}
    dy, dr = matrix(), matrix()

    def step():
        r, y = ar.residual_norm(x, **a)
        return (r, y, *ar.residual_norm_backward(dy, dr, x, r, **back))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(step(), want))
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
    # other values in the same places
    x.copy_(x.flip(0))
    graph.replay()
    again = step()
    assert all(torch.equal(p, q) for p, q in zip(out, again)) and not torch.equal(again[1], want[1])


def test_on_another_stream(ar):
    x, a, _ = inputs(13, 64, 1000, BF16, residual=True)
    want = ar.residual_norm(x, **a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r, y = ar.residual_norm(x, **a, stream=s)
    s.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(y, want[1])


def test_refusals(ar):
    x, a, matrix = inputs(17, 6, 32, BF16, residual=True)
    w, r = a["weight"], a["residual"]
    for bad, what in ((dict(), "weight or after_weight"), (dict(weight=w, bias=w.float()), "bias must be 32"),
                      (dict(weight=w[:31]), "weight must be 32"), (dict(after_weight=w, bias=w), "bias needs weight"),
                      (dict(weight=w, after_bias=w), "after_bias needs"), (dict(weight=w, gate=matrix()[:4]), "do not divide"),
                      (dict(weight=w, residual=r[:5]), "residual must be 6 x 32"), (dict(weight=w, eps=-1.0), "eps"),
                      (dict(weight=w, eps=float("nan")), "eps"), (dict(after_weight=w, y=matrix()), "y needs weight"),
                      (dict(weight=w, residual=r.float()), "residual must be a 2-D torch.bfloat16"),
                      (dict(weight=w, r=matrix().t()), "r must be 6 x 32")):
        with pytest.raises(ValueError, match=what):
            ar.residual_norm(x, **bad)
    for args, what in (((None, x, x, r, w), "dy and weight"), ((x, x, None, r, w, None, w), "needs x"),
                       ((x, x, None, None, w), "weight needs r"), ((x, x, x, None, w, None, w), "weight needs r"),
                       ((x, x[:3], x, r, w), "dr must be 6 x 32")):
        with pytest.raises(ValueError, match=what):
            ar.residual_norm_backward(*args)
    with pytest.raises(TypeError):
        ar.residual_norm_backward(None, None, x, r, w)


def test_inputs_that_require_grad_warn(ar):
    x, a, _ = inputs(19, 4, 16, BF16)
    with pytest.warns(UserWarning, match="weight requires grad"):
        ar.residual_norm(x, weight=a["weight"].clone().requires_grad_())
