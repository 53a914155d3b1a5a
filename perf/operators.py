"""The feed-forward operators as they are measured: their cases, their plain forms and their values in 64 bits.

Around the sum over ranks that this framework computes stand, in a tensor-parallel layer, the shard of the gated feed-forward
block before it (in training with its gradients, in serving with a down projection in 8-bit integers) and the dropout with the
residual after it.  A case is a dict; ``op`` says which operator it runs:

  ffn        h = act(x Wg^T) * (x Wu^T), with the two pre-activations returned where ``save`` is set (training)
  ffn_grad   its backward pass from the saved pre-activations: dx, dWg, dWu
  dropout    y = residual + dropout(x), the mask drawn from a counter-based generator and never stored
  dropout_grad   dx of it, the mask drawn again
  linear_i8  y = sx sw (q W^T) in 8-bit integers, scales for each token and channel; ``dynamic``: x is 16-bit and is quantised first
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One token of one sequence through one rank's shard: the latency of a decoding step; two weight matrices are streamed.
        {"name": "ffn decode 1", "op": "ffn", "M": 1, "K": 8192, "F": 3584, "dtype": "bf16", "act": "silu", "save": False},
        # A small serving batch whose size is no power of two.
        {"name": "ffn decode 13", "op": "ffn", "M": 13, "K": 5120, "F": 2048, "dtype": "fp16", "act": "gelu", "save": False},
        # The 440 x 5120 activations of the allreduce benchmark, with a shard that is no multiple of a tile.
        {"name": "ffn 440", "op": "ffn", "M": 440, "K": 5120, "F": 1736, "dtype": "bf16", "act": "silu", "save": False},
        # Training forward at 8192 tokens, pre-activations kept for the backward pass.
        {"name": "ffn train 8192", "op": "ffn", "M": 8192, "K": 8192, "F": 3584, "dtype": "bf16", "act": "silu", "save": True},
        # Gradients for a short micro-batch at the benchmark's 512 x 8192.
        {"name": "ffn grad 512", "op": "ffn_grad", "M": 512, "K": 8192, "F": 3584, "dtype": "bf16", "act": "silu"},
        # Gradients where nothing is aligned: rows of odd length, ragged tiles on every side.
        {"name": "ffn grad odd", "op": "ffn_grad", "M": 1001, "K": 1031, "F": 777, "dtype": "fp16", "act": "gelu"},
        # One token after the sum: launch latency.
        {"name": "dropout 1", "op": "dropout", "rows": 1, "cols": 5120, "pad": 0, "dtype": "bf16", "p": 0.1, "offset": 0},
        # A training batch after the sum; 32-bit element counters would still do, the mask's bits are the cost.
        {"name": "dropout 16384", "op": "dropout", "rows": 16384, "cols": 8192, "pad": 0, "dtype": "bf16", "p": 0.1, "offset": 0},
        # Gradient of a rank's block in a padded buffer; its elements begin past 2^32 in the whole tensor, at an odd place.
        {"name": "dropout grad 680", "op": "dropout_grad", "rows": 680, "cols": 5120, "pad": 40, "dtype": "fp32", "p": 0.5, "offset": (1 << 33) + 3},
        # One token through an 8-bit down projection, quantised on the way in.
        {"name": "linear_i8 decode 1", "op": "linear_i8", "M": 1, "K": 3584, "N": 8192, "dtype": "bf16", "dynamic": True},
        # The 440 x 5120 activations: a rank's 8-bit partial product that the allreduce sums.
        {"name": "linear_i8 440", "op": "linear_i8", "M": 440, "K": 2048, "N": 5120, "dtype": "bf16", "dynamic": True},
        # Prefill of a long prompt on activations that are 8-bit already.
        {"name": "linear_i8 4096", "op": "linear_i8", "M": 4096, "K": 8192, "N": 8192, "dtype": "fp16", "dynamic": False},
    ]


def draw(rng):
    def size(low, high, odd=0.4):
        n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        if rng.random() >= odd and n >= 64:
            n = n // 16 * 16
        return max(low, min(high, n))

    op = rng.choice(["ffn", "ffn", "ffn_grad", "dropout", "dropout_grad", "linear_i8"])
    half = rng.choice(["bf16", "fp16"])
    if op == "ffn":
        return {"op": op, "M": size(1, 8192), "K": size(64, 8192), "F": size(64, 3584), "dtype": half,
                "act": rng.choice(["silu", "gelu"]), "save": rng.random() < 0.5}
    if op == "ffn_grad":
        return {"op": op, "M": size(1, 4096), "K": size(64, 8192), "F": size(64, 3584), "dtype": half, "act": rng.choice(["silu", "gelu"])}
    if op == "linear_i8":
        return {"op": op, "M": size(1, 4096), "K": size(64, 8192), "N": size(64, 8192), "dtype": half, "dynamic": rng.random() < 0.5}
    return {"op": op, "rows": size(1, 16384), "cols": size(64, 8192), "pad": rng.choice([0, 0, 8, 5]), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "p": rng.choice([0.0, 0.1, 0.3, 0.5]), "offset": rng.choice([0, rng.randrange(1 << 20), rng.randrange(1 << 40)])}


# --------------------------------------------------------------------------------------------------------------- inputs

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op in ("ffn", "ffn_grad"):
        M, K, F = case["M"], case["K"], case["F"]
        s["x"] = _normal(gen, (M, K), dtype)
        s["wg"] = _normal(gen, (F, K), dtype, K ** -0.5)
        s["wu"] = _normal(gen, (F, K), dtype, K ** -0.5)
        if op == "ffn_grad":
            s["gate"] = (s["x"].float() @ s["wg"].float().T).to(dtype)
            s["up"] = (s["x"].float() @ s["wu"].float().T).to(dtype)
            s["dh"] = _normal(gen, (M, F), dtype)
        if own:
            from shot_allreduce_ranks_gb300 import GatedFFN
            s["ffn"] = GatedFFN(M, K, F, dtype=dtype, activation=case["act"], train=op == "ffn_grad")
    elif op in ("dropout", "dropout_grad"):
        rows, cols, wide = case["rows"], case["cols"], case["cols"] + case["pad"]
        s["x"] = _normal(gen, (rows, wide), dtype)[:, :cols]
        if op == "dropout":
            s["residual"] = _normal(gen, (rows, wide), dtype)[:, :cols]
        s["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=torch.Generator().manual_seed(int(seed))).item())
        s["sequence"] = 5 + int(seed) % 1000
    else:
        M, K, N = case["M"], case["K"], case["N"]
        if case["dynamic"]:
            s["x"] = _normal(gen, (M, K), dtype)
        else:
            s["q"] = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
            s["sx"] = torch.rand(M, generator=gen, device="cuda") * 0.02 + 0.005
        s["w"] = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
        s["sw"] = (torch.rand(N, generator=gen, device="cuda") + 0.5) / (73.0 * K ** 0.5)
    return s


# ------------------------------------------------------------------------------------------------------------------ run

def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case["op"], case, state)


def _run_own(op, c, s):
    import shot_allreduce_ranks_gb300 as ar

    if op == "ffn":
        return s["ffn"].forward(s["x"], s["wg"], s["wu"], save=c["save"])
    if op == "ffn_grad":
        return s["ffn"].backward(s["x"], s["wg"], s["wu"], s["gate"], s["up"], s["dh"])
    if op == "dropout":
        return ar.dropout(s["x"], c["p"], s["seed"], sequence=s["sequence"], offset=c["offset"], residual=s["residual"])
    if op == "dropout_grad":
        return ar.dropout_backward(s["x"], c["p"], s["seed"], sequence=s["sequence"], offset=c["offset"])
    if c["dynamic"]:
        q, sx = ar.quantize_rows(s["x"])
        return q, sx, ar.linear_i8(q, sx, s["w"], s["sw"], dtype=DTYPES[c["dtype"]])
    return ar.linear_i8(s["q"], s["sx"], s["w"], s["sw"], dtype=DTYPES[c["dtype"]])


GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def _act(v, act):
    """The activation and its derivative."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-v))
        return v * sig, sig * (1.0 + v * (1.0 - sig))
    t = torch.tanh(GELU_C * (v + GELU_A * v * v * v))
    return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * v * v)


def _philox_torch(first, n, seed, sequence, device):
    """The 32-bit draws of elements first .. first + n - 1 (Philox4x32, ten rounds: Salmon, Moraes, Dror, Shaw, 2011) in int64 arithmetic."""
    mask = 0xFFFFFFFF
    at = torch.arange(first // 4, (first + n - 1) // 4 + 1, dtype=torch.int64, device=device)
    c0, c1 = at & mask, at >> 32
    c2, c3 = torch.full_like(at, sequence & mask), torch.full_like(at, sequence >> 32)
    k0, k1 = seed & mask, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & mask) ^ c1 ^ k0, b & mask, ((a >> 32) & mask) ^ c3 ^ k1, a & mask
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return torch.stack((c0, c1, c2, c3), dim=1).reshape(-1)[first % 4: first % 4 + n]


def _run_plain(op, c, s):
    dtype = DTYPES[c["dtype"]]
    if op == "ffn":
        x = s["x"].float()
        g, u = x @ s["wg"].float().T, x @ s["wu"].float().T
        h = (_act(g, c["act"])[0] * u).to(dtype)
        return (h, g.to(dtype), u.to(dtype)) if c["save"] else h
    if op == "ffn_grad":
        x, wg, wu, dh = (s[k].float() for k in ("x", "wg", "wu", "dh"))
        f, df = _act(s["gate"].float(), c["act"])
        dg, du = dh * s["up"].float() * df, dh * f
        return (dg @ wg + du @ wu).to(dtype), (dg.T @ x).to(dtype), (du.T @ x).to(dtype)
    if op in ("dropout", "dropout_grad"):
        x = s["x"].float()
        keep = _philox_torch(c["offset"], x.numel(), s["seed"], s["sequence"], x.device) >= round(c["p"] * 2 ** 32)
        y = torch.where(keep.reshape(x.shape), x * (1.0 / (1.0 - c["p"])), torch.zeros((), device=x.device))
        return (y + s["residual"].float() if op == "dropout" else y).to(dtype)
    if c["dynamic"]:
        x = s["x"].float()
        top = x.abs().amax(dim=1)
        sx = top / torch.full_like(top, 127.0)
        q = torch.round(x / torch.where(sx > 0, sx, torch.ones_like(sx))[:, None])
    else:
        q, sx = s["q"].float(), s["sx"]
    y = ((q @ s["w"].float().T) * sx[:, None] * s["sw"][None, :]).to(dtype)
    return (q.to(torch.int8), sx, y) if c["dynamic"] else y


# -------------------------------------------------------------------------------------------------- the values in 64 bits

def _draws_numpy(first, n, seed, sequence):
    """The draws of elements first .. first + n - 1, block by block of counters, in unsigned 64-bit arithmetic on the host."""
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    b0, b1 = first >> 2, (first + n - 1 >> 2) + 1
    out = np.empty((b1 - b0, 4), dtype=np.uint32)
    for i in range(b0, b1, 1 << 16):
        at = np.arange(i, min(i + (1 << 16), b1), dtype=np.uint64)
        x = [at & low, at >> sh, np.full_like(at, sequence & 0xFFFFFFFF), np.full_like(at, sequence >> 32)]
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for r in range(10):
            p0, p1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            kr = [np.uint64((key[0] + r * 0x9E3779B9) % (1 << 32)), np.uint64((key[1] + r * 0xBB67AE85) % (1 << 32))]
            x = [(p1 >> sh) ^ x[1] ^ kr[0], p1 & low, (p0 >> sh) ^ x[3] ^ kr[1], p0 & low]
        for j in range(4):
            out[i - b0: i - b0 + len(at), j] = x[j]
    return out.reshape(-1)[first & 3: (first & 3) + n]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op in ("ffn", "ffn_grad"):
        if op == "ffn":
            z, v = torch.mm(d["x"], d["wg"].t()), torch.mm(d["x"], d["wu"].t())
        else:
            z, v = d["gate"], d["up"]
        if case["act"] == "silu":
            sig = torch.sigmoid(z)
            f, slope = z * sig, sig + z * sig * torch.sigmoid(-z)
        else:
            # 0.5 (1 + tanh t) is the logistic function of 2 t
            sig = torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
            f, slope = z * sig, sig + z * sig * (1.0 - sig) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * z ** 2)
        if op == "ffn":
            return (f * v, z, v) if case["save"] else f * v
        a, b = d["dh"] * v * slope, d["dh"] * f
        return torch.mm(torch.cat((a, b), 1), torch.cat((d["wg"], d["wu"]), 0)), torch.mm(a.t(), d["x"]), torch.mm(b.t(), d["x"])
    if op in ("dropout", "dropout_grad"):
        x = s["x"]
        bits = _draws_numpy(case["offset"], x.numel(), s["seed"], s["sequence"])
        kept = torch.from_numpy(bits >= np.uint32(round(case["p"] * 2 ** 32))).reshape(x.shape).to(x.device)
        y = torch.where(kept, d["x"] / (1.0 - case["p"]), 0.0)
        return y + d["residual"] if op == "dropout" else y
    if case["dynamic"]:
        # The integers are what the definition in 32 bits gives (a division rounded once, ties to even); they are compared with
        # the plain form's as whole numbers, so only the scale and the product have a value here.
        x32 = s["x"].to(torch.float32).cpu().numpy()
        top = np.abs(x32).max(axis=1)
        scale = np.divide(top, np.float32(127.0), dtype=np.float32)
        q = np.rint(np.divide(x32, np.where(scale > 0, scale, np.float32(1.0))[:, None], dtype=np.float32))
        q = torch.from_numpy(q).to("cuda").double()
        sx = torch.from_numpy(scale).to("cuda").double()
    else:
        q, sx = d["q"], d["sx"]
    y = torch.mm(q, d["w"].t()) * (sx[:, None] * d["sw"][None, :])
    return (None, d["x"].abs().amax(1) / 127.0, y) if case["dynamic"] else y


# ----------------------------------------------------------------------------------------------------------------- work

def work(case):
    op, e = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op in ("dropout", "dropout_grad"):
        n = case["rows"] * case["cols"]
        return {"bytes": (3 if op == "dropout" else 2) * n * e, "flops": 2 * n}
    M, K = case["M"], case["K"]
    if op == "linear_i8":
        N = case["N"]
        # x in 8 bits, or in 16 bits and written in 8; the weights; the output; the scales.
        x = M * K * (3 if case["dynamic"] else 1)
        return {"bytes": x + N * K + 2 * M * N + 4 * (M + N), "flops": 2 * M * K * N}
    F = case["F"]
    if op == "ffn":
        return {"bytes": e * (M * K + 2 * F * K + M * F * (3 if case["save"] else 1)), "flops": 4 * M * K * F}
    return {"bytes": e * (2 * M * K + 4 * F * K + 3 * M * F), "flops": 8 * M * K * F}
