"""A layer's steps around the feed-forward block from their definitions in 64 bits, with bounds on what a right kernel
may be off, for the tests.

Bounds are first-order sums of the roundings on the way, E = 2^-24 being half a step of fp32 relative to the value.  A
sum over a row is made by at least 32 threads (256 above 2,048 columns), each adding its own elements one by one, and
joined by at most 10 further additions, so a partial sum passes through at most depth(cols) roundings.  A sum over rows
is made by up to 200 CTAs or more, each over its own rows, and their parts by sixteen warps one by one.
"""
import torch

E = 2.0 ** -24


def depth(cols):
    return min(cols / 32, 64 + cols / 256) + 16


def depth_rows(rows):
    return min(rows, rows / 200 + 64)


def hat(v, ev, kind, eps):
    """(normalised rows, their bound, factor, its relative bound) of rows that are off by at most ev."""
    n = depth(v.shape[1])
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    emean = ev.mean(1, keepdim=True) + (n + 2) * E * v.abs().mean(1, keepdim=True) if kind == "layer" else 0.0
    d = v - mean
    ed = ev + emean + E * d.abs()
    ms = d.square().mean(1, keepdim=True)
    ems = (n + 6) * E * ms + 2 * (d.abs() * ed).mean(1, keepdim=True) + ed.square().mean(1, keepdim=True)
    f = (ms + eps) ** -0.5
    rel = 0.5 * ems / (ms + eps) + 4 * E
    h = d * f
    return h, ed * f + h.abs() * (rel + 2 * E), f, rel


class Norm:
    """One call's arguments in 64 bits; None for what is absent."""

    def __init__(self, x=None, residual=None, weight=None, bias=None, after_weight=None, after_bias=None, gate=None,
                 kind="rms", eps=1e-6, residual_scale=1.0, weight_offset=0.0):
        self.kind, self.eps, self.alpha, self.offset = kind, eps, residual_scale, weight_offset
        for name, t in (("x", x), ("residual", residual), ("weight", weight), ("bias", bias), ("aw", after_weight),
                        ("ab", after_bias), ("gate", gate)):
            setattr(self, name, None if t is None else t.double())

    def affine(self, h, eh, weight, bias):
        w = self.offset + weight
        v, e = h * w, eh * w.abs() + 3 * E * (h * w).abs() + E * h.abs() * (abs(self.offset) + weight.abs())
        return (v, e) if bias is None else (v + bias, e + E * (v + bias).abs())

    def gates(self, rows):
        return None if self.gate is None else self.gate.repeat_interleave(rows // self.gate.shape[0], 0)

    def branch(self):
        """(z, its bound)"""
        if self.aw is None:
            return self.x, torch.zeros_like(self.x)
        h, eh, _, _ = hat(self.x, torch.zeros_like(self.x), self.kind, self.eps)
        return self.affine(h, eh, self.aw, self.ab)

    def forward(self):
        """((r, its bound), (y, its bound) or None), without the final rounding."""
        r, er = self.branch()
        if self.gate is not None:
            g = self.gates(len(r))
            r, er = r * g, er * g.abs() + 2 * E * (r * g).abs()
        if self.residual is not None:
            add = self.alpha * self.residual
            er = er + 3 * E * (r.abs() + add.abs())
            r = r + add
        if self.weight is None:
            return (r, er), None
        h, eh, _, _ = hat(r, er, self.kind, self.eps)
        return (r, er), self.affine(h, eh, self.weight, self.bias)

    def through(self, d, ed, v):
        """Gradient of norm(v) * w + b with respect to v where d, within ed, is that of norm(v); (norm(v), its bound) too."""
        n = depth(v.shape[1])
        h, eh, f, rel = hat(v, torch.zeros_like(v), self.kind, self.eps)

        def mean(t, e):
            return t.mean(1, keepdim=True), e.mean(1, keepdim=True) + (n + 3) * E * t.abs().mean(1, keepdim=True)

        m1, em1 = mean(d * h, d.abs() * eh + ed * h.abs())
        m0, em0 = mean(d, ed) if self.kind == "layer" else (torch.zeros_like(m1), torch.zeros_like(m1))
        t = d - m0 - h * m1
        et = ed + em0 + eh * m1.abs() + h.abs() * em1 + 4 * E * (d.abs() + m0.abs() + (h * m1).abs())
        return f * t, f * et + (f * t).abs() * (rel + 2 * E), h, eh

    def backward(self, dy, dr, r):
        """{name: (gradient, its bound)} without the final rounding; r is the stored one."""
        like = dy if dy is not None else dr
        rows = len(like)
        n = depth_rows(rows)
        g = torch.zeros(like.shape, dtype=torch.float64, device=like.device) if dr is None else dr.double()
        eg = torch.zeros_like(g)
        out = {}

        def total(v, e, k=1):
            """Sums over each of k runs of rows."""
            v, e = v.reshape(k, -1, v.shape[1]), e.reshape(k, -1, v.shape[1])
            return v.sum(1), e.sum(1) + n * E * v.abs().sum(1)

        if dy is not None:
            dy, w = dy.double(), self.offset + self.weight
            d = dy * w
            t, et, h, eh = self.through(d, 2 * E * d.abs() + E * dy.abs() * (abs(self.offset) + self.weight.abs()), r.double())
            eg = eg + et + 2 * E * (g.abs() + t.abs())
            g = g + t
            out["dweight"] = [v[0] for v in total(dy * h, dy.abs() * eh + E * (dy * h).abs())]
            if self.bias is not None:
                out["dbias"] = [v[0] for v in total(dy, torch.zeros_like(dy))]
        out["dresidual"] = (self.alpha * g, abs(self.alpha) * eg + 2 * E * (self.alpha * g).abs())
        if self.gate is not None:
            z, ez = self.branch()
            out["dgate"] = total(g * z, eg * z.abs() + (g.abs() + eg) * ez + E * (g * z).abs(), len(self.gate))
            a = self.gates(rows)
            g, eg = g * a, eg * a.abs() + E * (g * a).abs()
        if self.aw is not None:
            d = g * (self.offset + self.aw)
            ed = eg * (self.offset + self.aw).abs() + 2 * E * d.abs() + E * g.abs() * (abs(self.offset) + self.aw.abs())
            t, et, h, eh = self.through(d, ed, self.x)
            out["dafter_weight"] = [v[0] for v in total(g * h, eg * h.abs() + (g.abs() + eg) * eh + E * (g * h).abs())]
            if self.ab is not None:
                out["dafter_bias"] = [v[0] for v in total(g, eg)]
            g, eg = t, et
        out["dx"] = (g, eg)
        return out


def routing(logits, top_k, normalize):
    """(experts, weights in 64 bits, relative bound on the weights) by the definition, on the host."""
    z = logits.double().cpu()
    T, n = z.shape
    expert = torch.full((T, top_k), -1, dtype=torch.int32)
    weight = torch.zeros((T, top_k), dtype=torch.float64)
    bound = torch.zeros((T, 1), dtype=torch.float64)
    for t in range(T):
        def place(e):
            v = float(z[t, e])
            return (0, 0.0, e) if v != v else (1, -v, e)

        best = [e for e in sorted(range(n), key=place)[:top_k] if float(z[t, e]) != -float("inf")]
        if not best:
            continue
        expert[t, :len(best)] = torch.tensor(best, dtype=torch.int32)
        d = z[t, best] - z[t, best[0]]
        p = torch.exp(d)
        weight[t, :len(best)] = p / (p.sum() if normalize else torch.exp(z[t] - z[t, best[0]]).sum())
        # the difference's rounding moves the exponential by |d| E, which is itself good to 2 units (4 E); as much again
        # for the sum, whose terms count by their size (d e^d <= 1/e each), its additions, and the division
        bound[t] = (2 * d.abs().nan_to_num(0, 0, 0).max() + 16 + n / 32 + 10) * E
    return expert, weight, bound


def moe(x, logits, w_gate, w_up, w_down, top_k, activation="silu", normalize=True, first_expert=0):
    """(out, its bound without the final rounding, experts, weights, the weights' bound)"""
    from tests import ff_reference as ff
    u, tiny = ff.U[x.dtype], ff.TINY[x.dtype]
    expert, weight, rel = routing(logits, top_k, normalize)
    K, F = x.shape[1], w_gate.shape[1]
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    bound, size = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(w_gate.shape[0]):
        t, j = torch.nonzero(expert == first_expert + e, as_tuple=True)
        if not len(t):
            continue
        w, ew = weight[t, j].to(x.device)[:, None], (weight[t, j] * rel[t, 0]).to(x.device)[:, None]
        t = t.to(x.device)
        (h, _, _), (eh, _, _) = ff.forward(x[t], w_gate[e], w_up[e], activation)
        eh = eh + u * (h.abs() + eh) + tiny
        d = w_down[e].double()
        part, epart = h @ d.T, (eh + F * ff.E32 * (h.abs() + eh)) @ d.abs().T
        out[t] += w * part
        bound[t] += w * epart + ew * (part.abs() + epart)
        size[t] += w * (part.abs() + epart)
    # the weighted pieces are added one by one: at most a piece for every 64 inner columns of a token's experts
    return out, bound + (top_k * (F / 64 + 1) + 10) * E * size, expert, weight, weight * rel


def quantize_i4(w, group, zero):
    """(q, scale, zero point or None) by the definition: IEEE fp32, the scale rounded to 16 bits before it divides."""
    N, K = w.shape
    groups = -(-K // group)
    v = torch.zeros((N, groups * group), device=w.device)
    v[:, :K] = w.float()
    v = v.view(N, groups, group)
    seven, fifteen = torch.tensor(7.0, device=w.device), torch.tensor(15.0, device=w.device)
    high, low = v.amax(2).clamp_min(0), v.amin(2).clamp_max(0)
    want = high / fifteen - low / fifteen if zero else torch.maximum(high, -low) / seven
    bad = ~torch.isfinite(v).all(2)
    scale = torch.where(bad, float("nan"), want).to(w.dtype)
    none = (scale == 0) | bad
    by = torch.where(none, 1.0, scale.float())
    z = torch.where(none, 0.0, torch.round(-low / by).clamp_max(15)) if zero else torch.full_like(by, 8.0)
    q = (torch.round(v / by[:, :, None]) + z[:, :, None]).clamp(0.0 if zero else 1.0, 15.0)
    q = torch.where(none[:, :, None], z[:, :, None].clamp_min(0.0 if zero else 1.0), q)
    return q.reshape(N, -1)[:, :K].to(torch.uint8), scale, z.to(torch.uint8) if zero else None


def weights_i4(q, scale, zero, group):
    """The weights in 64 bits."""
    def spread(t):
        return t.double().repeat_interleave(group, 1)[:, :q.shape[1]]

    return (q.double() - (8.0 if zero is None else spread(zero))) * spread(scale)
