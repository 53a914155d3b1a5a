"""The feed-forward operators on the GPU against their definitions in 64 bits.

Every limit comes from tests/ff_reference.py: derived from the operators'
roundings, not from what the kernels gave.
"""
import numpy as np
import pytest
import torch

from shot_allreduce_ranks_gb300 import build
from tests import ff_reference as ref

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


class Framed:
    """A matrix inside a larger allocation of a marker value, with `pad` columns
    after each row and `shift` elements before the first: reads past it bring the
    marker (NaN) into the result, writes past it are found by intact()."""

    def __init__(self, rows, cols, dtype, pad=0, shift=0, fill=None):
        self.ld = cols + pad
        mark = float("nan") if dtype.is_floating_point else 77
        self.buf = torch.full((64 + shift + (rows + 3) * self.ld + 64,), mark, dtype=dtype, device=DEV)
        self.t = self.buf[64 + shift:][:(rows + 2) * self.ld].view(rows + 2, self.ld)[:rows, :cols]
        if fill is not None:
            self.t.copy_(fill)

    def intact(self):
        n = self.buf.numel() - self.t.numel()
        b = self.buf.clone()
        start = self.t.storage_offset()
        view = torch.as_strided(b, self.t.shape, self.t.stride(), start)
        zero = float("nan") if b.is_floating_point() else 77
        view.fill_(zero)
        same = torch.isnan(b) if b.is_floating_point() else b == 77
        return bool(same.all()) and n > 0


def frame(t, pad, shift):
    return Framed(t.shape[0], t.shape[1], t.dtype, pad, shift, t)


def normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


# (M, K, F): one of everything, tile edges on each side, ragged, deep, and more tiles than SMs.
SIZES = [(1, 1, 1), (1, 64, 8), (2, 7, 3), (8, 8, 8), (1, 512, 96), (3, 1000, 40), (13, 136, 264),
         (17, 129, 33), (33, 256, 128), (63, 64, 65), (64, 72, 64), (65, 2048, 136), (127, 192, 129),
         (128, 128, 128), (129, 136, 120), (200, 512, 392), (257, 1096, 512)]
LAYOUTS = [(0, 0), (8, 0), (5, 0), (0, 1), (3, 3)]  # (pad, shift): aligned, padded, odd rows, odd base


def run_forward(ar, M, K, F, dtype, act, pad, shift, seed=0):
    g = gen(seed)
    x, wg, wu = normal(g, (M, K), dtype), normal(g, (F, K), dtype, K ** -0.5), normal(g, (F, K), dtype, K ** -0.5)
    fx, fg, fu = (frame(t, pad, shift) for t in (x, wg, wu))
    outs = [Framed(M, F, dtype, pad, shift) for _ in range(3)]
    with ar.GatedFFN(M, K, F, dtype=dtype, activation=act) as ffn:
        got = ffn.forward(fx.t, fg.t, fu.t, out=outs[0].t, gate=outs[1].t, up=outs[2].t)
        alone = ffn.forward(fx.t, fg.t, fu.t)
        torch.cuda.synchronize()
    want, bounds = ref.forward(x, wg, wu, act)
    for a, b, e, what in zip(got, want, bounds, ("out", "gate", "up")):
        ref.assert_close(a, b, e, what)
    assert torch.equal(alone, got[0])
    assert all(f.intact() for f in outs)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype,act", [(BF16, "silu"), (FP16, "gelu")])
def test_forward_sizes(ar, size, dtype, act):
    run_forward(ar, *size, dtype, act, 0, 0)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", [(1, 264, 72), (13, 136, 264), (30, 2056, 72), (6, 1040, 40), (150, 264, 200)])
@pytest.mark.parametrize("dtype,act", [(BF16, "gelu"), (FP16, "silu")])
def test_forward_layouts(ar, size, layout, dtype, act):
    run_forward(ar, *size, dtype, act, *layout, seed=1)


@pytest.mark.parametrize("size", [(1030, 520, 3000), (2100, 128, 1400), (130, 8192, 256), (1, 8192, 512),
                                  # the split of k over a cluster: whole, in two, in four, and fewer tokens than it is made for
                                  (20, 2048, 2100), (9, 8192, 1032), (100, 4096, 4000), (128, 2056, 10000), (33, 520, 2048),
                                  (65, 72, 2048), (128, 4160, 1288)])
def test_forward_many_tiles_and_deep_sums(ar, size):
    run_forward(ar, *size, BF16, "silu", 0, 0, seed=2)


def run_backward(ar, M, K, F, dtype, act, pad, shift, seed=0, **need):
    g = gen(seed)
    x, wg, wu = normal(g, (M, K), dtype), normal(g, (F, K), dtype, K ** -0.5), normal(g, (F, K), dtype, K ** -0.5)
    gate, up, dout = normal(g, (M, F), dtype), normal(g, (M, F), dtype), normal(g, (M, F), dtype)
    ins = [frame(t, pad, shift) for t in (x, wg, wu, gate, up, dout)]
    shapes = [(M, K), (F, K), (F, K)]
    wanted = [need.get("need_dx", True)] + 2 * [need.get("need_dw", True)]
    outs = [Framed(*s, dtype, pad, shift) for s in shapes]
    with ar.GatedFFN(M + 3, K, F, dtype=dtype, activation=act, train=True) as ffn:
        got = ffn.backward(*(f.t for f in ins), *(f.t if w else None for f, w in zip(outs, wanted)), **need)
        torch.cuda.synchronize()
    want, bounds = ref.backward(x, wg, wu, gate, up, dout, act)
    for a, b, e, w, what in zip(got, want, bounds, wanted, ("dx", "dw_gate", "dw_up")):
        assert (a is not None) == w
        if w:
            ref.assert_close(a, b, e, what)
    assert all(f.intact() for f, w in zip(outs, wanted) if w)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype,act", [(BF16, "silu"), (FP16, "gelu")])
def test_backward_sizes(ar, size, dtype, act):
    run_backward(ar, *size, dtype, act, 0, 0)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", [(1, 264, 72), (150, 264, 200)])
def test_backward_layouts(ar, size, layout):
    run_backward(ar, *size, BF16, "gelu", *layout, seed=1)


@pytest.mark.parametrize("size", [(520, 1030, 700), (4100, 136, 136), (40, 2600, 1400)])
def test_backward_many_tiles_and_deep_sums(ar, size):
    run_backward(ar, *size, FP16, "silu", 0, 0, seed=2)


@pytest.mark.parametrize("M", [1, 15, 16, 17, 33, 64])
@pytest.mark.parametrize("K,F,dtype,act", [(136, 72, BF16, "silu"), (131, 77, FP16, "gelu"), (520, 1032, FP16, "silu")])
def test_gradients_of_a_few_tokens_in_two_parts(ar, M, K, F, dtype, act):
    """Up to 64 tokens dgate and dup reach the products in two 16-bit parts: what is
    left is the outputs' own rounding and the sums'."""
    g = gen(M + K)
    x, wg, wu = normal(g, (M, K), dtype), normal(g, (F, K), dtype, K ** -0.5), normal(g, (F, K), dtype, K ** -0.5)
    gate, up, dout = normal(g, (M, F), dtype), normal(g, (M, F), dtype), normal(g, (M, F), dtype)
    outs = [Framed(*s, dtype, 3, 1) for s in ((M, K), (F, K), (F, K))]
    with ar.GatedFFN(200, K, F, dtype=dtype, activation=act, train=True) as ffn:
        # the workspace holds another call's values first
        big = normal(g, (200, F), dtype, float("inf"))
        ffn.backward(normal(g, (200, K), dtype), wg, wu, big, big, big)
        got = ffn.backward(x, wg, wu, gate, up, dout, *(f.t for f in outs))
    want, bounds = ref.backward(x, wg, wu, gate, up, dout, act, two_parts=True)
    for a, b, e, what in zip(got, want, bounds, ("dx", "dw_gate", "dw_up")):
        ref.assert_close(a, b, e, what)
    assert all(f.intact() for f in outs)


def test_backward_parts(ar):
    run_backward(ar, 70, 72, 136, BF16, "silu", 0, 0, need_dx=False)
    run_backward(ar, 70, 72, 136, BF16, "silu", 0, 0, need_dw=False)


def test_no_tokens(ar):
    with ar.GatedFFN(4, 24, 16, train=True) as ffn:
        x, w = torch.zeros(0, 24, dtype=BF16, device=DEV), torch.ones(16, 24, dtype=BF16, device=DEV)
        assert ffn.forward(x, w, w).shape == (0, 16)
        e = torch.zeros(0, 16, dtype=BF16, device=DEV)
        full = [torch.full((16, 24), 3.0, dtype=BF16, device=DEV) for _ in range(2)]
        dx, dwg, dwu = ffn.backward(x, w, w, e, e, e, None, *full)
        assert dx.shape == (0, 24) and not dwg.any() and not dwu.any()
    e = torch.zeros(0, 8, dtype=BF16, device=DEV)
    assert ar.dropout(e, 0.5, 1).shape == (0, 8)
    q, s = ar.quantize_rows(e)
    assert ar.linear_i8(q, s, torch.ones(4, 8, dtype=torch.int8, device=DEV), torch.ones(4, device=DEV)).shape == (0, 4)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_gradients_against_differences(ar, act, dtype):
    """Directional derivatives of the 64-bit loss by central differences, on
    inputs whose pre-activations the 16-bit types hold exactly."""
    g, (M, K, F) = gen(11), (40, 16, 24)
    x = torch.randint(-2, 3, (M, K), generator=g, device=DEV).to(dtype) / 2
    wg, wu = (torch.randint(-1, 2, (F, K), generator=g, device=DEV).to(dtype) / 2 for _ in range(2))
    dout = normal(g, (M, F), dtype)
    with ar.GatedFFN(M, K, F, dtype=dtype, activation=act, train=True) as ffn:
        _, gate, up = ffn.forward(x, wg, wu, save=True)
        grads = ffn.backward(x, wg, wu, gate, up, dout)
    assert torch.equal(gate.double(), x.double() @ wg.double().T)
    _, bounds = ref.backward(x, wg, wu, gate, up, dout, act)
    vals = [t.double() for t in (x, wg, wu)]

    def loss(x, wg, wu):
        return float((ref.activation(x @ wg.T, act)[0] * (x @ wu.T) * dout.double()).sum())

    for k in range(3):
        d = torch.randn(vals[k].shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-5
        moved = [vals[:k] + [vals[k] + s * h * d] + vals[k + 1:] for s in (1, -1)]
        slope = (loss(*moved[0]) - loss(*moved[1])) / (2 * h)
        got = grads[k].double()
        limit = ((bounds[k] + ref.U[dtype] * (got.abs() + bounds[k])) * d.abs()).sum() + 1e-6 * (got * d).abs().sum()
        assert abs(float((got * d).sum()) - slope) <= float(limit)


@pytest.mark.parametrize("size", [(5, 64, 40), (50, 264, 200), (40, 2048, 1032), (140, 136, 72)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_values_stay_in_their_rows(ar, size, bad):
    M, K, F = size
    g = gen(5)
    x, wg, wu = normal(g, (M, K), BF16), normal(g, (F, K), BF16, 0.1), normal(g, (F, K), BF16, 0.1)
    dout = normal(g, (M, F), BF16)
    row = M - 2
    with ar.GatedFFN(M, K, F, train=True) as ffn:
        clean = ffn.forward(x, wg, wu, save=True)
        dclean = ffn.backward(x, wg, wu, clean[1], clean[2], dout)
        x2 = x.clone()
        x2[row, K // 2] = bad
        got = ffn.forward(x2, wg, wu, save=True)
        dgot = ffn.backward(x2, wg, wu, got[1], got[2], dout)
    others = torch.arange(M, device=DEV) != row
    for a, b in zip(got + dgot[:1], clean + dclean[:1]):
        assert torch.equal(a[others], b[others])
    assert not torch.isfinite(got[1][row]).any()
    assert torch.isnan(dgot[0][row]).any() or torch.isinf(dgot[0][row]).any()


def test_large_preactivations(ar):
    """Pre-activations far out on both sides: the sigmoid is 0 or 1 and nothing overflows on the way."""
    big = torch.tensor([-3e4, -200.0, -90.0, -30.0, 0.0, 30.0, 90.0, 200.0, 3e4], device=DEV)
    for act in ("silu", "gelu"):
        x = big[:, None].to(BF16).expand(9, 8).contiguous()
        w = torch.zeros(16, 8, dtype=BF16, device=DEV)
        w[:, 0] = 1
        with ar.GatedFFN(9, 8, 16, activation=act, train=True) as ffn:
            out, gate, up = ffn.forward(x, w, w, save=True)
            grads = ffn.backward(x, w, w, gate, up, torch.ones_like(out))
        want, bounds = ref.forward(x, w, w, act)
        ref.assert_close(out, want[0], bounds[0], act)
        want, bounds = ref.backward(x, w, w, gate, up, torch.ones_like(out), act)
        for a, b, e in zip(grads, want, bounds):
            ref.assert_close(a, b, e, act + " gradient")


def test_rows_past_2_31_elements(ar):
    """Rows whose offsets in elements pass 31 bits, in the input and in the output."""
    M, ld, K, F = 140, (1 << 24) + 8, 64, 40
    buf = torch.zeros(M * ld, dtype=BF16, device=DEV)
    x = buf.view(M, ld)[:, :K]
    g = gen(6)
    x.copy_(normal(g, (M, K), BF16))
    wg, wu = normal(g, (F, K), BF16, 0.1), normal(g, (F, K), BF16, 0.1)
    out = buf.view(M, ld)[:, 128:128 + F]
    with ar.GatedFFN(M, K, F) as ffn:
        ffn.forward(x, wg, wu, out=out)
    want, bounds = ref.forward(x, wg, wu, "silu")
    ref.assert_close(out, want[0], bounds[0], "out")
    y = ar.dropout(x, 0.25, 3, out=out[:, :0].new_empty(M, K))
    v, e = ref.dropout(x.contiguous(), 0.25, 3, 0, 0)
    ref.assert_close(y, v, e, "dropout")


# ------------------------------------------------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols,pad,shift", [
    (1, 1, 0, 0), (1, 8, 0, 0), (3, 5, 0, 0), (7, 64, 8, 0), (5, 129, 7, 0), (4, 100, 3, 1), (65, 257, 0, 0),
    (33, 96, 0, 1), (300, 40, 16, 0)])
@pytest.mark.parametrize("p,offset", [(0.1, 0), (0.5, (1 << 33) + 3), (0.25, 6), (0.3, (1 << 34) - 40)])
def test_dropout(ar, dtype, rows, cols, pad, shift, p, offset):
    g = gen(rows * 1000 + cols)
    x, r = normal(g, (rows, cols), dtype), normal(g, (rows, cols), dtype)
    fx, fr, fo, fd = frame(x, pad, shift), frame(r, pad, shift), Framed(rows, cols, dtype, pad, shift), Framed(rows, cols, dtype, pad, shift)
    seed, sequence = 0x9E3779B97F4A7C15, (1 << 40) + 77
    y = ar.dropout(fx.t, p, seed, sequence, offset, residual=fr.t, out=fo.t)
    dx = ar.dropout_backward(fx.t, p, seed, sequence, offset, dx=fd.t)
    want, bound = ref.dropout(x, p, seed, sequence, offset, r)
    ref.assert_close(y, want, bound, "forward")
    want, bound = ref.dropout(x, p, seed, sequence, offset)
    ref.assert_close(dx, want, bound, "backward")
    assert torch.equal(dx == 0, (want == 0) | (x == 0))
    assert fo.intact() and fd.intact()


def test_dropout_gradient_against_differences(ar):
    """The operator is linear in x: the change of the loss is the gradient times the change."""
    g = gen(4)
    x, dx_dir, dy = (torch.randint(-8, 9, (30, 72), generator=g, device=DEV).float() for _ in range(3))
    y0, y1 = (ar.dropout(v, 0.5, 9, 2).double() for v in (x, x + dx_dir))
    grad = ar.dropout_backward(dy, 0.5, 9, 2).double()
    # integers times 1 / (1 - 0.5) = 2 are exact
    assert float(((y1 - y0) * dy.double()).sum()) == float((grad * dx_dir.double()).sum())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_dropout_of_none_and_of_all(ar, dtype):
    x, r = normal(gen(1), (9, 77), dtype), normal(gen(2), (9, 77), dtype)
    assert torch.equal(ar.dropout(x, 0.0, 5), x)
    assert torch.equal(ar.dropout(x, 1.0, 5, residual=r), r)
    assert not ar.dropout(x, 1.0, 5).any()


def test_dropped_elements_that_are_not_finite_count_as_zero(ar):
    x = torch.full((16, 128), float("nan"), device=DEV)
    r = torch.ones(16, 128, device=DEV)
    y = ar.dropout(x, 0.5, 8, residual=r)
    keep = torch.from_numpy(ref.draws(0, 2048, 8, 0) >= 2 ** 31).view(16, 128).to(DEV)
    assert torch.equal(torch.isnan(y), keep) and bool((y[~keep] == 1).all())


def test_dropout_in_place_and_in_blocks(ar):
    x, r = normal(gen(1), (64, 200), BF16), normal(gen(2), (64, 200), BF16)
    whole = ar.dropout(x, 0.3, 21, 4, residual=r)
    for into in (x.clone(), r.clone()):
        a, b = (into, r) if torch.equal(into, x) else (x, into)
        assert torch.equal(ar.dropout(a, 0.3, 21, 4, residual=b, out=into), whole)
    # the blocks of a reduce-scatter over 8 ranks draw the whole tensor's mask
    parts = [ar.dropout(x[8 * k:8 * k + 8], 0.3, 21, 4, offset=8 * k * 200, residual=r[8 * k:8 * k + 8]) for k in range(8)]
    assert torch.equal(torch.cat(parts), whole)
    assert not torch.equal(ar.dropout(x, 0.3, 21, 5, residual=r), whole)
    assert not torch.equal(ar.dropout(x, 0.3, 22, 4, residual=r), whole)


def test_dropout_past_2_31_elements(ar):
    n = (1 << 31) + 4104
    x = torch.ones(1, n, dtype=BF16, device=DEV)
    y = ar.dropout(x, 0.5, 77)
    tail = ar.dropout(x[:, :4096], 0.5, 77, offset=n - 4096)
    assert torch.equal(y[:, -4096:], tail)
    keep = torch.from_numpy(ref.draws(n - 4096, 4096, 77, 0) >= 2 ** 31).to(DEV)
    assert torch.equal(tail[0] != 0, keep)
    # 2^31 draws of a fair coin: the mean is within 6 / (2 sqrt(2^31))
    assert abs(float((y != 0).sum()) / n - 0.5) < 6 / (2 * 2 ** 15.5)


# ---------------------------------------------------------------------------------------------------------- 8-bit product

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (1, 3584, 0, 0), (5, 77, 3, 1), (40, 2048, 0, 0), (300, 264, 8, 0), (2, 40000, 0, 0), (3, 8192, 0, 0), (3, 8200, 0, 0),
                                                    (4, 4097, 7, 0), (1, 2051, 0, 0), (1700, 512, 0, 0), (1333, 2048, 16, 0),
                                                    (1301, 2057, 7, 0), (1310, 96, 0, 0), (1305, 13, 3, 0), (1900, 1000, 5, 1)])
def test_quantize_rows(ar, dtype, rows, cols, pad, shift):
    x = normal(gen(rows + cols), (rows, cols), dtype)
    if rows > 1:
        x[1] = 0
    q, s = Framed(rows, cols, torch.int8, pad, shift), torch.empty(rows, device=DEV)
    ar.quantize_rows(frame(x, pad, shift).t, q=q.t, scale=s)
    want_q, want_s = ref.quantize(x)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.t.cpu().numpy(), want_q)
    assert q.intact()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_quantize_rows_near_halves_and_far_scales(ar, dtype):
    """Quotients that fall on and next to halves, and scales from the smallest
    normal numbers up: the integers are those of an IEEE division."""
    k = torch.arange(-127, 128, device=DEV).float()
    rows = [torch.cat([k, k + 0.5, k - 0.5 + 2.0 ** -12, k + 0.5 - 2.0 ** -12, k / 127]).clamp(-127, 127) * f
            for f in (1.0, 3.0, 0.1, 1 / 3, 2.0 ** -10, 7e4 / 127)]
    x = torch.stack(rows + [normal(gen(s), (5 * 255,), FP32) * 2.0 ** e for s, e in ((1, 0), (2, -12), (3, 9))])
    if dtype is not FP16:
        x = torch.cat([x, x * 2.0 ** -99, x * 2.0 ** -110, x * 2.0 ** 100])
    x = x.to(dtype)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    q, s = ar.quantize_rows(x)
    want_q, want_s = ref.quantize(x)
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)


def test_quantize_rows_that_are_not_finite(ar):
    x = normal(gen(3), (6, 300), FP32)
    x[1, 7], x[2, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    x[5] = 2.0 ** -149  # a scale that underflows to zero
    q, s = ar.quantize_rows(x)
    assert torch.isnan(s[1]) and torch.isinf(s[2]) and torch.isinf(s[4]) and s[5] == 0
    assert not q[[1, 2, 4, 5]].any()
    want_q, want_s = ref.quantize(x[[0, 3]])
    assert np.array_equal(q[[0, 3]].cpu().numpy(), want_q) and np.array_equal(s[[0, 3]].cpu().numpy(), want_s)
    y = ar.linear_i8(q, s, torch.ones(16, 300, dtype=torch.int8, device=DEV), torch.ones(16, device=DEV))
    assert torch.isnan(y[[1, 2, 4]]).all() and torch.isfinite(y[[0, 3, 5]]).all()


def run_i8(ar, M, K, N, dtype, pad=0, shift=0, full=False, seed=0):
    g = gen(seed + M + K + N)
    x = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    if full:  # the largest sums there are
        x.fill_(-128)
        w.fill_(-128)
    sx = torch.rand(M, generator=g, device=DEV) + 0.5
    sw = (torch.rand(N, generator=g, device=DEV) + 0.5) * (1e-3 / K ** 0.5)
    out = Framed(M, N, dtype, pad, shift)
    ar.linear_i8(frame(x, pad, shift).t, sx, frame(w, pad, shift).t, sw, out=out.t)
    total = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    scale = sx.double()[:, None] * sw.double()[None, :]
    # sums are exact while every partial sum fits 24 bits, whatever the order
    off = torch.where(mag <= 2.0 ** 24, 0.0, K * ref.E32 * mag)
    ref.assert_close(out.t, total * scale, off * scale + 2 * ref.E32 * (total * scale).abs(), "linear_i8")
    assert out.intact()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_linear_i8_sizes(ar, size, dtype):
    run_i8(ar, *size, dtype)


@pytest.mark.parametrize("layout", [(0, 0), (16, 0), (8, 0), (5, 0), (0, 1), (3, 3), (0, 8), (1, 15)])
@pytest.mark.parametrize("size", [(1, 272, 72), (9, 272, 72), (30, 2064, 72), (6, 4112, 40), (70, 272, 200), (150, 272, 200)])
def test_linear_i8_layouts(ar, size, layout):
    run_i8(ar, *size, BF16, *layout)


@pytest.mark.parametrize("size", [(1030, 528, 3000), (130, 8192, 264), (1, 8192, 1000), (16, 4096, 200)])
def test_linear_i8_many_tiles_and_deep_sums(ar, size):
    run_i8(ar, *size, FP16)


@pytest.mark.parametrize("size", [(1, 1024, 40), (12, 1024, 40), (150, 1024, 200), (1, 4096, 40), (150, 4096, 72)])
def test_linear_i8_largest_sums(ar, size):
    run_i8(ar, *size, BF16, full=True)


@pytest.mark.parametrize("size", [(4096, 8192, 8192), (1030, 8192, 2600), (440, 2048, 5120), (64, 3584, 8192)])
def test_linear_i8_the_same_bits_every_time(ar, size):
    """Many launches, half of them beside copies on another stream.  A sum of K products of numbers up to 127 that vary has a
    standard deviation of 5376 sqrt(K) < 2^19, so that all partial sums fit 24 bits by 30 of them: the sums are
    exact, and with two products in fp32 and one rounding so are the results' bits."""
    M, K, N = size
    g = gen(M + N)
    x = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sx = torch.rand(M, generator=g, device=DEV) + 0.5
    sw = (torch.rand(N, generator=g, device=DEV) + 0.5) * (1e-3 / K ** 0.5)
    want = ((x.double() @ w.double().T).float() * sx[:, None] * sw[None, :]).half()
    side, room = torch.cuda.Stream(), torch.empty(2, 1 << 26, device=DEV, dtype=torch.uint8)
    torch.cuda.synchronize()
    for k in range(80):
        if k % 2:
            with torch.cuda.stream(side):
                for _ in range(1 + k % 5):
                    room[0].copy_(room[1])
        assert torch.equal(ar.linear_i8(x, sx, w, sw, dtype=FP16), want), "launch %d" % k
    torch.cuda.synchronize()


@pytest.mark.parametrize("size", [(4096, 8192, 3584), (1000, 2056, 520)])
def test_large_products_have_the_same_bits_every_time(ar, size):
    M, K, F = size
    t, ffn = inputs(M, K, F, 3), ar.GatedFFN(M, K, F, dtype=BF16, train=True)
    first = everything(ar, ffn, t)
    for _ in range(20):
        for a, b in zip(first, everything(ar, ffn, t)):
            assert torch.equal(a, b)


# --------------------------------------------------------------------------------------------------- how they are called

def everything(ar, ffn, t, stream=None):
    out, gate, up = ffn.forward(t["x"], t["wg"], t["wu"], save=True, stream=stream)
    grads = ffn.backward(t["x"], t["wg"], t["wu"], gate, up, t["dout"], stream=stream)
    y = ar.dropout(out, 0.2, 5, residual=gate, stream=stream)
    q, s = ar.quantize_rows(y, stream=stream)
    return (out, gate, up, *grads, y, q, s, ar.linear_i8(q, s, t["w8"], t["s8"], stream=stream))


def inputs(M, K, F, seed):
    g = gen(seed)
    return {"x": normal(g, (M, K), BF16), "wg": normal(g, (F, K), BF16, K ** -0.5), "wu": normal(g, (F, K), BF16, K ** -0.5),
            "dout": normal(g, (M, F), BF16), "w8": torch.randint(-127, 128, (K, F), generator=g, device=DEV, dtype=torch.int8),
            "s8": torch.rand(K, generator=g, device=DEV)}


@pytest.mark.parametrize("M", [4, 200])
def test_streams_graphs_and_repetition(ar, M):
    """The same bits on the current stream, on another one, and from a replayed graph whose inputs change."""
    K, F = 256, 272
    sets = [inputs(M, K, F, s) for s in (1, 2)]
    with ar.GatedFFN(M, K, F, train=True) as ffn:
        want = [everything(ar, ffn, t) for t in sets]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            other = everything(ar, ffn, sets[0])
        given = everything(ar, ffn, sets[0], stream=side)
        side.synchronize()
        live = {k: v.clone() for k, v in sets[0].items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = everything(ar, ffn, live)
        for t, w in zip(sets, want):
            for k, v in t.items():
                live[k].copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(captured, w))
        assert all(torch.equal(a, b) for a, b in zip(other, want[0]))
        assert all(torch.equal(a, b) for a, b in zip(given, want[0]))


@pytest.mark.parametrize("M,K,F", [(24, 2048, 1032), (100, 4096, 1032), (700, 1032, 2600), (300, 777, 501)])
def test_many_calls_give_the_same_bits(ar, M, K, F):
    """Hundreds of calls back to back, several tiles to a CTA: a stage reused too
    early or a sum read too soon would show as a difference."""
    t = inputs(M, K, F, 3)
    with ar.GatedFFN(M, K, F, train=True) as ffn:
        want = everything(ar, ffn, t)
        off = torch.zeros((), dtype=torch.int64, device=DEV)
        for _ in range(150):
            for a, b in zip(everything(ar, ffn, t), want):
                off += (a != b).sum()
    assert int(off) == 0
    assert ar.ops_device_status() == 0


def test_scratch_is_optional_at_the_c_entry(ar):
    """Unaligned operands without scratch take another kernel, with too little they are refused."""
    from shot_allreduce_ranks_gb300 import _lib
    lib, (M, K, N) = ar.load(), (150, 131, 72)
    g = gen(8)
    x = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sx, sw = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
    outs = [torch.empty(M, N, dtype=FP16, device=DEV) for _ in range(2)]
    need = lib.ar_linear_i8_scratch_bytes(x.data_ptr(), K, w.data_ptr(), K, M, K, N)
    scratch = torch.empty(need, dtype=torch.uint8, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    for out, p, n, want in ((outs[0], None, 0, _lib.AR_OK), (outs[1], scratch.data_ptr(), need, _lib.AR_OK),
                            (outs[1], scratch.data_ptr(), need - 1, _lib.AR_ERR_INVALID_ARG)):
        assert lib.ar_linear_i8(x.data_ptr(), K, sx.data_ptr(), w.data_ptr(), K, sw.data_ptr(), out.data_ptr(), N, M, K, N,
                                _lib.AR_FP16, p, n, s) == want
    assert torch.equal(*outs)  # sums of integers below 2^24 are exact in either
    x, wg, wu = normal(g, (M, K), BF16), normal(g, (N, K), BF16, 0.1), normal(g, (N, K), BF16, 0.1)
    gate, up, dout = normal(g, (M, N), BF16), normal(g, (M, N), BF16), normal(g, (M, N), BF16)
    with ar.GatedFFN(M, K, N, train=True) as ffn:
        out = torch.empty(M, N, dtype=BF16, device=DEV)
        assert lib.ar_ffn_forward(ffn._h, x.data_ptr(), K, wg.data_ptr(), wu.data_ptr(), K, out.data_ptr(), None, None, N,
                                  M, None, 0, s) == _lib.AR_OK
        want, bounds = ref.forward(x, wg, wu, "silu")
        ref.assert_close(out, want[0], bounds[0], "forward")
        grads = [torch.empty(a, K, dtype=BF16, device=DEV) for a in (M, N, N)]
        ptrs = [t.data_ptr() for t in grads]
        assert lib.ar_ffn_backward(ffn._h, x.data_ptr(), K, wg.data_ptr(), wu.data_ptr(), K, gate.data_ptr(), up.data_ptr(),
                                   dout.data_ptr(), N, ptrs[0], K, ptrs[1], ptrs[2], K, M, None, 0, s) == _lib.AR_OK
        want, bounds = ref.backward(x, wg, wu, gate, up, dout, "silu")
        for a, b, e in zip(grads, want, bounds):
            ref.assert_close(a, b, e, "backward")


def test_python_refusals(ar):
    x, w = torch.zeros(4, 16, dtype=BF16, device=DEV), torch.zeros(8, 16, dtype=BF16, device=DEV)
    h = torch.zeros(4, 8, dtype=BF16, device=DEV)
    with ar.GatedFFN(4, 16, 8) as ffn:
        for bad in ((x.to(FP16), w, w), (x[:, :8], w, w), (x, w[:4], w), (x, w.T, w), (x.cpu(), w, w), (x[0], w, w)):
            with pytest.raises(ValueError):
                ffn.forward(*bad)
        with pytest.raises(ValueError, match="together"):
            ffn.forward(x, w, w, gate=h)
        with pytest.raises(ar.ArError):  # made without the workspace
            ffn.backward(x, w, w, h, h, h)
    with ar.GatedFFN(2, 16, 8, train=True) as ffn, pytest.raises(ValueError, match="workspace"):
        ffn.backward(x, w, w, h, h, h)
    with pytest.raises(ar.ArError):
        ar.dropout(x, 1.5, 0)
    with pytest.raises(ValueError):
        ar.dropout(x, 0.5, -1)
    with pytest.raises(ValueError):
        ar.dropout(x, 0.5, 0, residual=h)
    with pytest.raises(ValueError):
        ar.quantize_rows(x.to(torch.int8))
    q, s = ar.quantize_rows(x)
    with pytest.raises(ValueError):
        ar.linear_i8(q, s, q[:, :8], s)
    with pytest.raises(ValueError):
        ar.linear_i8(q, s[:2], q, s)
    with pytest.raises(ValueError):
        ar.linear_i8(q, s, q, s, dtype=FP32)
