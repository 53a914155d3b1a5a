"""A layer of experts dealt out to virtual ranks, served, and a gated block between norms, trained.

Serving: every rank holds a part of the experts and all of the router's logits; its partial outputs are
summed by the allreduce, after which the norms, the residual and a projection with 4-bit weights follow:

    r, y    = residual_norm(x, residual)                 the norm before the experts
    part_e  = moe_ffn(y, logits, rank's experts)         zeros for tokens whose experts are elsewhere
    s       = sum over ranks of part                     AllReduce
    r2, y2  = residual_norm(s, r, gate, norm after it)   both norms around the residual
    z       = linear_i4(y2, W)                           4-bit weights

Training: y = norm(a residual + gate norm(x) wa) w through a gated feed-forward shard and back, every
gradient of it.

Run it on a GPU:  python examples/expert_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from shot_allreduce_ranks_gb300 import (AllReduce, GatedFFN, linear_i4, moe_ffn, quantize_i4,  # noqa: E402
                                        residual_norm, residual_norm_backward)


def make(shape, scale=1.0, mean=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + mean).bfloat16()


class Served:
    """The weights of R ranks: E / R experts each, and what every rank has."""

    def __init__(self, ranks=4, experts=16, top_k=3, hidden=1024, width=264, out=520, tokens=13):
        self.ranks, self.local, self.top_k = ranks, experts // ranks, top_k
        self.router = make((experts, hidden), hidden ** -0.5, seed=1)
        self.w_gate = make((experts, width, hidden), hidden ** -0.5, seed=2)
        self.w_up = make((experts, width, hidden), hidden ** -0.5, seed=3)
        self.w_down = make((experts, hidden, width), width ** -0.5, seed=4)
        self.before, self.after, self.last = (make((hidden,), 0.1, 1.0, seed=s) for s in (5, 6, 7))
        self.gate = make((1, hidden), 0.1, 0.5, seed=8)
        self.w_out = make((out, hidden), hidden ** -0.5, seed=9)
        self.w_out_i4 = quantize_i4(self.w_out, group=64)
        self.allreduce = AllReduce(ranks, tokens * hidden)
        # The sum's buffers stay where they are, so that its pointer tables are made once (a captured step needs that).
        self.parts, self.sums = ([torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]
                                 for _ in range(2))

    def step(self, x, residual):
        """(experts chosen, z): one decoding step of all tokens."""
        r, y = residual_norm(x, residual, self.before)
        logits = y.float() @ self.router.float().T
        for k in range(self.ranks):
            mine = slice(k * self.local, (k + 1) * self.local)
            _, chosen, _ = moe_ffn(y, logits, self.w_gate[mine], self.w_up[mine], self.w_down[mine], self.top_k,
                                   first_expert=k * self.local, out=self.parts[k], routing=True)
        s = self.allreduce(self.parts, self.sums)[0]
        _, y2 = residual_norm(s, r, self.last, after_weight=self.after, gate=self.gate, residual_scale=0.9)
        return chosen, linear_i4(y2, self.w_out_i4)

    def reference(self, x, residual, chosen):
        """The same layer in 64 bits, unsharded, with the experts that were chosen (near a border the
        16-bit activations choose)."""
        def norm(v, w):
            return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()

        r = x.double() + residual.double()
        y = norm(r, self.before)
        logits = y @ self.router.double().T
        share = torch.softmax(logits.gather(1, chosen.long()), 1)
        s = torch.zeros_like(y)
        for j in range(self.top_k):
            e = chosen[:, j].long()
            g = torch.einsum("tk,tfk->tf", y, self.w_gate[e].double())
            h = torch.nn.functional.silu(g) * torch.einsum("tk,tfk->tf", y, self.w_up[e].double())
            s += share[:, j:j + 1] * torch.einsum("tf,tkf->tk", h, self.w_down[e].double())
        r2 = 0.9 * r + self.gate.double() * norm(s, self.after)
        return norm(r2, self.last) @ self.w_out_i4.dequantize().double().T


def training_step(tokens=200, hidden=520, width=136, seed=20):
    """(gradients of x, residual, weight, after_weight, gate, w_gate, w_up) and the same by torch's differentiation in 64 bits."""
    x, residual, dh, dr = (make((tokens, hidden if i != 2 else width), seed=seed + i) for i in range(4))
    w, wa = make((hidden,), 0.1, 1.0, seed=seed + 4), make((hidden,), 0.1, 1.0, seed=seed + 5)
    gate, wg, wu = make((1, hidden), 0.2, 0.5, seed=seed + 6), make((width, hidden), 0.05, seed=seed + 7), make((width, hidden), 0.05, seed=seed + 8)
    norm = dict(after_weight=wa, gate=gate, residual_scale=0.7)
    with GatedFFN(tokens, hidden, width, train=True) as ffn:
        r, y = residual_norm(x, residual, w, **norm)
        _, g, u = ffn.forward(y, wg, wu, save=True)
        dy, dwg, dwu = ffn.backward(y, wg, wu, g, u, dh)
        dx, dres, dw, _, dwa, _, dgate = residual_norm_backward(dy, dr, x, r, w, **norm)
    p = [t.double().requires_grad_() for t in (x, residual, w, wa, gate, wg, wu)]

    def rms(v):
        return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt()

    rr = 0.7 * p[1] + p[4] * (rms(p[0]) * p[3])
    yy = rms(rr) * p[2]
    h = torch.nn.functional.silu(yy @ p[5].T) * (yy @ p[6].T)
    torch.autograd.backward((h, rr), (dh.double(), dr.double()))
    return (dx, dres, dw, dwa, dgate, dwg, dwu), [t.grad for t in p]


def off(got, want):
    """2-norm of the difference over 2-norm of the value."""
    return float((got.double() - want).norm() / want.norm())


def main(say=print):
    layer = Served()
    x, residual = make((13, 1024), seed=30), make((13, 1024), 2.0, seed=31)
    chosen, z = layer.step(x, residual)
    found = {"served": off(z, layer.reference(x, residual, chosen))}
    layer.allreduce.close()
    got, want = training_step()
    names = ("dx", "dresidual", "dweight", "dafter_weight", "dgate", "dw_gate", "dw_up")
    found.update({k: off(a, b) for k, a, b in zip(names, got, want)})
    for k, v in found.items():
        say("%-14s %.2e" % (k, v))
    return found


if __name__ == "__main__":
    main()
