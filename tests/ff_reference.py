"""The feed-forward operators from their definitions in 64 bits, with bounds on
what a right kernel may be off, for the tests.

Bounds.  u is the unit roundoff of the 16-bit type (half a unit in the last
place: 2^-8 for bfloat16, 2^-11 for float16) and `tiny` half its smallest
subnormal.  A sum of n exact products in fp32, in any order and with additions
that may truncate, is within n 2^-23 of the sum of the products' absolute
values.  A sigmoid from the fast exponential is within (8 + 2 |s|) 2^-23 of
its value in relative terms (the exponential's documented 2 + 1.2 |s| units,
and a few for the addition and the division).
"""
import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E32 = 2.0 ** -23


def activation(v, act):
    """(f, f', bound on f as computed in fp32, bound on f')."""
    if act == "silu":
        s, ds = v, torch.ones_like(v)
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s, ds = c * (v + 0.044715 * v ** 3), c * (1.0 + 3 * 0.044715 * v ** 2)
    sig = torch.sigmoid(s)
    rel = (8 + 2 * s.abs()) * E32
    f = v * sig
    df = sig + v * sig * torch.sigmoid(-s) * ds
    # sig (1 + v (1 - sig) ds): each term's rounding, and 1 - sig off by rel * sig
    edf = 4 * rel * sig * (1.0 + (v * ds).abs())
    return f, df, 2 * rel * f.abs() + 1e-37, edf + 1e-37


def forward(x, wg, wu, act):
    """((out, gate, up), their bounds without the final rounding)."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    n = x.shape[1] * E32
    g, u = x @ wg.T, x @ wu.T
    eg, eu = n * (x.abs() @ wg.abs().T), n * (x.abs() @ wu.abs().T)
    f, _, ef, _ = activation(g, act)
    ef = ef + 1.13 * eg  # |f'| <= 1.13 for both activations
    h = f * u
    return (h, g, u), (ef * u.abs() + f.abs() * eu + ef * eu + E32 * h.abs(), eg, eu)


def backward(x, wg, wu, gate, up, dout, act, two_parts=False):
    """((dx, dwg, dwu), their bounds without the final rounding).

    two_parts: the pre-activations' gradients are held as the sum of two 16-bit
    numbers, so that what remains of their rounding is its square.
    """
    r, tiny = U[x.dtype], TINY[x.dtype]
    r = r * r if two_parts else r
    x, wg, wu, gate, up, dout = (t.double() for t in (x, wg, wu, gate, up, dout))
    f, df, ef, edf = activation(gate, act)
    a, b = dout * up * df, dout * f
    ea = (dout * up).abs() * (edf + 2 * E32 * df.abs())
    eb = dout.abs() * (ef + E32 * f.abs())
    ea, eb = ea + r * (a.abs() + ea) + tiny, eb + r * (b.abs() + eb) + tiny  # rounded to 16 bits
    aa, ab = a.abs() + ea, b.abs() + eb
    dx = a @ wg + b @ wu
    edx = ea @ wg.abs() + eb @ wu.abs() + 2 * a.shape[1] * E32 * (aa @ wg.abs() + ab @ wu.abs())
    n = a.shape[0] * E32
    return ((dx, a.T @ x, b.T @ x),
            (edx, ea.T @ x.abs() + n * (aa.T @ x.abs()), eb.T @ x.abs() + n * (ab.T @ x.abs())))


def assert_close(got, want, bound, what=""):
    """|got - want| <= bound, and one rounding to got's type of a value within it."""
    limit = bound + U[got.dtype] * (want.abs() + bound) + TINY[got.dtype]
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all(), "%s: not finite" % what
    bad = off > limit
    if bad.any():
        at = int(torch.argmax((off / limit).flatten()))
        raise AssertionError("%s: %d of %d off; worst at %d: got %.9g want %.9g, limit %.3g" % (
            what, int(bad.sum()), bad.numel(), at, got.flatten()[at], want.flatten()[at], limit.flatten()[at]))


def draws(first, n, seed, sequence):
    """The 32-bit draws of elements first .. first + n - 1 in Python integers' arithmetic, vectorised."""
    b0 = first >> 2
    blocks = np.array([b0 + i for i in range(((first + n - 1) >> 2) - b0 + 1)], dtype=object)
    c = [blocks & 0xFFFFFFFF, blocks >> 32, blocks * 0 + (sequence & 0xFFFFFFFF), blocks * 0 + (sequence >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, axis=1).reshape(-1).astype(np.uint64)
    return words[first & 3: (first & 3) + n]


def dropout(x, p, seed, sequence, offset, residual=None):
    """(value in 64 bits, bound without the final rounding)."""
    keep = torch.from_numpy(draws(offset, x.numel(), seed, sequence) >= round(p * 2 ** 32))
    keep = keep.reshape(x.shape).to(x.device)
    kept = torch.where(keep, x.double() / (1.0 - p) if p < 1 else 0.0, 0.0)
    if residual is None:
        return kept, 2 * E32 * kept.abs()
    return kept + residual.double(), 2 * E32 * kept.abs() + E32 * (kept + residual.double()).abs()


def quantize(x):
    """(q, scale) by the definition: IEEE fp32 divisions, ties to even."""
    v = x.float().cpu().numpy()
    top = np.abs(v).max(axis=1)
    scale = np.divide(top, np.float32(127), dtype=np.float32)
    by = np.where(scale > 0, scale, np.float32(1))
    with np.errstate(invalid="ignore"):
        q = np.rint(np.divide(v, by[:, None], dtype=np.float32))
    q[~np.isfinite(top)] = 0
    return np.clip(q, -127, 127).astype(np.int8), scale
