"""A tensor-parallel feed-forward layer over virtual ranks, in training and in serving.

Every rank holds the whole activations x, a shard of the gated projections
(rows of Wgate and Wup) and the matching columns of the down projection:

    h_r    = act(x Wgate_r^T) * (x Wup_r^T)          GatedFFN, one kernel
    part_r = h_r Wdown_r^T                           a plain matrix product, or linear_i8 in serving
    s      = sum over r of part_r                    AllReduce
    y      = x + dropout(s)                          dropout: every rank draws the same mask

and in training the gradients the same way back; dx is a second sum over the
ranks.  ``training_step`` also takes the sum as a reduce-scatter, where rank r
keeps a block of tokens and draws its part of the mask by the block's place.

Run it on a GPU:  python examples/tensor_parallel_feed_forward.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from shot_allreduce_ranks_gb300 import (AllReduce, GatedFFN, dropout, dropout_backward,  # noqa: E402
                                        linear_i8, quantize_rows)


class Layer:
    """R ranks' shards of one layer, and what the calls need."""

    def __init__(self, ranks: int, tokens: int, hidden: int, width: int, p: float = 0.1, seed: int = 1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(rows, cols, scale):
            return (torch.randn(rows, cols, generator=g, device="cuda") * scale).bfloat16()

        self.ranks, self.tokens, self.hidden, self.width, self.p = ranks, tokens, hidden, width, p
        self.w_gate = [normal(width, hidden, hidden ** -0.5) for _ in range(ranks)]
        self.w_up = [normal(width, hidden, hidden ** -0.5) for _ in range(ranks)]
        self.w_down = [normal(hidden, width, (ranks * width) ** -0.5) for _ in range(ranks)]
        self.w_down_i8 = [quantize_rows(w) for w in self.w_down]  # one scale for each output channel
        self.ffn = [GatedFFN(tokens, hidden, width, train=True) for _ in range(ranks)]
        self.allreduce = AllReduce(ranks, tokens * hidden)

    def close(self):
        for f in self.ffn:
            f.close()
        self.allreduce.close()

    def sum(self, parts):
        return [t.view_as(parts[0]) for t in self.allreduce([t.reshape(-1) for t in parts])]


def training_step(layer: Layer, x, dy, seed: int, step: int):
    """Outputs of every rank and the gradients: (y, y by blocks, dx, [dWgate], [dWup], [dWdown])."""
    R, p = layer.ranks, layer.p
    saved, parts = [], []
    for r in range(R):
        saved.append(layer.ffn[r].forward(x, layer.w_gate[r], layer.w_up[r], save=True))
        parts.append(saved[r][0] @ layer.w_down[r].T)
    sums = layer.sum(parts)
    y = [dropout(s, p, seed, sequence=step, residual=x) for s in sums]

    # The same with the tokens scattered: rank r's block begins at element r * rows * hidden.
    rows = layer.tokens // R
    blocks = layer.allreduce.reduce_scatter([t.reshape(-1) for t in parts], recvcount=rows * layer.hidden)
    y_blocks = [dropout(b.view(rows, -1), p, seed, sequence=step, offset=r * rows * layer.hidden,
                        residual=x[r * rows:(r + 1) * rows]) for r, b in enumerate(blocks)]

    ds = dropout_backward(dy, p, seed, sequence=step)
    dx_parts, dw_gate, dw_up, dw_down = [], [], [], []
    for r in range(R):
        h, gate, up = saved[r]
        dw_down.append(ds.T @ h)
        dx, dg, du = layer.ffn[r].backward(x, layer.w_gate[r], layer.w_up[r], gate, up, ds @ layer.w_down[r])
        dx_parts.append(dx)
        dw_gate.append(dg)
        dw_up.append(du)
    dx = layer.sum(dx_parts)[0] + dy  # the residual's path
    return y, torch.cat(y_blocks), dx, dw_gate, dw_up, dw_down


def serving_step(layer: Layer, x):
    """The layer's output with the down projection in 8-bit integers (no dropout)."""
    parts = []
    for r in range(layer.ranks):
        h = layer.ffn[r].forward(x, layer.w_gate[r], layer.w_up[r])
        q, scale = quantize_rows(h)
        parts.append(linear_i8(q, scale, *layer.w_down_i8[r]))
    return x + layer.sum(parts)[0]


def reference(layer: Layer, x, dy=None, keep=None):
    """The unsharded layer in 64 bits by torch's differentiation: (y, dx, [dWgate], [dWup], [dWdown]).

    ``keep``: the mask; None: no dropout, and only y is returned.
    """
    x = x.double().requires_grad_()
    ws = [[w.double().requires_grad_() for w in ws] for ws in (layer.w_gate, layer.w_up, layer.w_down)]
    s = sum((torch.nn.functional.silu(x @ g.T) * (x @ u.T)) @ d.T for g, u, d in zip(*ws))
    if keep is None:
        return (x + s).detach()
    y = x + s * keep / (1.0 - layer.p)
    y.backward(dy.double())
    return y.detach(), x.grad, *([w.grad for w in group] for group in ws)


def off(got, want):
    """2-norm of the difference over 2-norm of the value."""
    return float((got.double() - want).norm() / want.norm())


def main(ranks=4, tokens=440, hidden=5120, width=1736, seed=20, step=3, say=print):
    layer = Layer(ranks, tokens, hidden, width)
    g = torch.Generator(device="cuda").manual_seed(9)
    x, dy = (torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    y, y_blocks, dx, dw_gate, dw_up, dw_down = training_step(layer, x, dy, seed, step)
    # The mask, for the reference: ones through dropout.
    keep = (dropout(torch.ones_like(x, dtype=torch.float32), layer.p, seed, sequence=step) != 0).double()
    want = reference(layer, x, dy, keep)
    served = serving_step(layer, x)
    found = {
        "ranks agree": all(torch.equal(t, y[0]) for t in y),
        "blocks agree": torch.equal(y_blocks, y[0][:y_blocks.shape[0]]),
        "y": off(y[0], want[0]), "dx": off(dx, want[1]),
        "dw_gate": max(off(a, b) for a, b in zip(dw_gate, want[2])),
        "dw_up": max(off(a, b) for a, b in zip(dw_up, want[3])),
        "dw_down": max(off(a, b) for a, b in zip(dw_down, want[4])),
        "served": off(served, reference(layer, x)),
    }
    layer.close()
    for k, v in found.items():
        say("%-14s %s" % (k, v if isinstance(v, bool) else "%.2e" % v))
    return found


if __name__ == "__main__":
    main()
