"""The norms' kernels where a CTA, or a group of its threads, walks over many rows: its sums over them, the copies
ahead and their reuse, and gate rows that follow one another."""
import pytest
import torch

from shot_allreduce_ranks_gb300 import build
from tests import layer_reference as layer
from tests.ff_reference import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("dx", "dresidual", "dweight", "dbias", "dafter_weight", "dafter_bias", "dgate")


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def rows_walked(rows, cols, branch, gates, in_registers=True):
    """Rows that a group of threads takes one after the other, at least, as the backward pass deals them out."""
    parts = min(rows, 640 if cols <= 4096 else 320 if cols <= 8192 else 160)
    if in_registers:
        n = 8 if cols <= 8192 else 16
        threads = -(-cols // (32 * n)) * 32
        groups = max(1, 256 // threads)
        cta = threads * groups
        per_sm = 1 if cta > 512 or (branch and cta > 256) else (512 if branch else 1024) // cta
    else:
        groups, per_sm = 1, 2
    want = min(per_sm * sms(), parts)
    gates = max(gates, 1)
    if gates <= want:
        chunk = -(-(rows // gates) // (want // gates))
        return chunk // groups
    return gates // (want * groups) * (rows // gates)


def inputs(seed, rows, cols, dtype, residual=True, after=False, before=True, bias=False, gates=0, kind="rms", scale=1.0, offset=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, mean=0.0, size=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * size + mean).to(dtype)

    a = dict(kind=kind, eps=1e-5, residual_scale=scale, weight_offset=offset)
    x = normal(rows, cols, mean=0.3)
    if residual:
        a["residual"] = normal(rows, cols, size=2.0)
    for name, there in (("weight", before), ("after_weight", after)):
        if there:
            a[name] = normal(cols, mean=1.0 - offset, size=0.3)
            if bias:
                a[name.replace("weight", "bias")] = normal(cols)
    if gates:
        a["gate"] = normal(gates, cols)
    return x, a, normal


def check(ar, x, a, normal):
    (wr, er), y = layer.Norm(x, **a).forward()
    r, got = ar.residual_norm(x, **a)
    if r is not None:
        assert_close(r, wr, er, "r")
    if y is not None:
        assert_close(got, *y, "y")
    dy, dr = normal(*x.shape) if "weight" in a else None, normal(*x.shape) if r is not None else None
    back = {k: v for k, v in a.items() if k != "residual"}
    got = dict(zip(NAMES, ar.residual_norm_backward(dy, dr, x, r, **back)))
    want = layer.Norm(x, **a).backward(dy, dr, x if r is None else r)
    if r is None:
        del want["dresidual"]
    for k, v in want.items():
        assert_close(got[k], *v, k)


# Two groups of a CTA, one, one of 512 and of 1,024 threads, three of 64 and of 96; odd rows of the same.  Every ring is refilled and wraps.
@pytest.mark.parametrize("rows,cols", [(6200, 1024), (2800, 4096), (1300, 8192), (12000, 512), (7400, 640), (7400, 641), (2800, 4093), (5400, 1031)])
@pytest.mark.parametrize("kind,bias", [("rms", False), ("layer", True), ("rms", True), ("layer", False)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_plain(ar, rows, cols, kind, bias, dtype):
    assert rows_walked(rows, cols, False, 0) >= 4
    check(ar, *inputs(rows, rows, cols, dtype, kind=kind, bias=bias))


@pytest.mark.parametrize("rows,cols", [(2800, 1024), (1300, 4096), (1300, 2047)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_plain_fp32(ar, rows, cols, kind):
    assert rows_walked(rows, cols, False, 0) >= 2
    check(ar, *inputs(rows, rows, cols, FP32, kind=kind, bias=True, residual=False))


# The branch: 256, 512 and then each number of threads from 512 on at which a thread has other registers.
@pytest.mark.parametrize("rows,cols", [(1500, 2048), (900, 4096), (700, 5120), (700, 5376), (700, 5384), (700, 6144), (700, 6152), (700, 8192),
                                       (900, 2045), (700, 5119), (700, 5383), (700, 6143), (700, 6145), (700, 8191)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("parts", [dict(after=True), dict(after=True, bias=True, gates=1, kind="layer", scale=0.7, offset=1.0),
                                   dict(after=True, before=False, kind="layer"), dict(gates=2, residual=False)])
def test_branch(ar, rows, cols, dtype, parts):
    assert rows_walked(rows, cols, True, parts.get("gates", 0)) >= 3
    check(ar, *inputs(cols, rows, cols, dtype, **parts))


@pytest.mark.parametrize("rows,gates,cols", [(1600, 1600, 2048), (1600, 800, 2048), (700, 700, 5120), (900, 450, 4096), (700, 350, 5121),
                                             (9000, 4500, 512), (2800, 700, 2040)])
@pytest.mark.parametrize("kind,bias", [("rms", False), ("layer", True)])
def test_gate_rows_one_after_the_other(ar, rows, gates, cols, kind, bias):
    """Several whole gate rows to a group of threads."""
    run = rows // gates
    assert rows_walked(rows, cols, True, gates) >= 2 * run
    check(ar, *inputs(gates, rows, cols, BF16, after=True, bias=bias, gates=gates, kind=kind))
    check(ar, *inputs(gates, rows, cols, FP16, after=False, gates=gates, kind=kind))


@pytest.mark.parametrize("rows,cols", [(700, 9000), (700, 8193)])
@pytest.mark.parametrize("parts", [dict(bias=True, kind="layer"), dict(after=True, bias=True, gates=1, scale=0.5), dict(after=True, gates=350)])
def test_rows_read_again(ar, rows, cols, parts):
    assert rows_walked(rows, cols, True, parts.get("gates", 0), in_registers=False) >= 4
    check(ar, *inputs(cols, rows, cols, FP32, **parts))


@pytest.mark.parametrize("rows,cols", [(700, 12288), (700, 16384)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_wide_rows_in_registers(ar, rows, cols, kind):
    assert rows_walked(rows, cols, False, 0) >= 4
    check(ar, *inputs(cols, rows, cols, BF16, kind=kind, bias=True))


# Copied ahead by whole CTAs (2,432 and 304 at a time) and by warps (4,864).
@pytest.mark.parametrize("rows,cols", [(9000, 1024), (1600, 8192), (1600, 8184), (800, 16384), (20000, 256), (20000, 504)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("parts", [dict(), dict(after=True, bias=True, gates=1, kind="layer", scale=0.7), dict(residual=False, kind="layer"),
                                   dict(after=True, before=False), dict(gates=200, offset=1.0)])
def test_rows_copied_ahead(ar, rows, cols, dtype, parts):
    assert rows > 3 * sms() and cols % 8 == 0
    x, a, _ = inputs(cols, rows, cols, dtype, **parts)
    (wr, er), y = layer.Norm(x, **a).forward()
    r, got = ar.residual_norm(x, **a)
    if r is not None:
        assert_close(r, wr, er, "r")
    if y is not None:
        assert_close(got, *y, "y")
