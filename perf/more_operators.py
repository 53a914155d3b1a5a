"""More operators of a tensor-parallel layer as they are measured: their cases, their plain forms and their values in 64 bits.

They stand beside the feed-forward operators around the sum over ranks: the norms and the residual that follow the sum, the
product of a few tokens with 4-bit weights, and one rank's part of a mixture of gated feed-forward experts, whose partial
outputs the sum joins.  A case is a dict; ``op`` says which operator it runs:

  norm       r = residual_scale * residual + gate * norm(x) * wa,  y = norm(r) * w: the norm after a block, its gate, the
             residual and the norm before the next block, each but one of them optional
  norm_grad  its backward pass from x, the stored r and the gradients of y and r: of x, the residual, both weights, biases, gate
  linear_i4  y[m, n] = sum_k x[m, k] scale[n, k / group] (q[n, k] - zero[n, k / group]), q in 0 .. 15
  moe        y[t] = sum over a token's top_k experts of weight * Wdown (act(Wgate x) * (Wup x)), with the routing returned
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------- cases

def _norm_case(op, rows, cols, dtype, kind="rms", residual=True, after=False, before=True, bias=False, gates=0, scale=1.0, offset=0.0, pad=0):
    """gates: rows of the gate matrix, each for rows / gates rows (0: no gate)."""
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "kind": kind, "residual": residual, "after": after, "before": before,
            "bias": bias, "gates": gates, "scale": scale, "offset": offset, "pad": pad}


def listed():
    return [
        # One token after the sum: the residual is added and the next block's norm taken; launch latency.
        {"name": "norm 1", **_norm_case("norm", 1, 5120, "bf16")},
        # The 440 x 5120 activations of the allreduce benchmark, norms on both sides of the residual.
        {"name": "norm both 440", **_norm_case("norm", 440, 5120, "bf16", after=True, offset=1.0)},
        # Seven sequences of odd length and width, layer norms with biases, a gate for each sequence; nothing is aligned.
        {"name": "norm layer odd", **_norm_case("norm", 1001, 1031, "fp16", kind="layer", bias=True, gates=7, scale=0.81)},
        # A training batch.
        {"name": "norm 16384", **_norm_case("norm", 16384, 8192, "bf16")},
        # Gradients of a training batch.
        {"name": "norm grad 8192", **_norm_case("norm_grad", 8192, 8192, "bf16")},
        # Gradients of every part in 32 bits, rows in a padded buffer.
        {"name": "norm grad all 680", **_norm_case("norm_grad", 680, 5120, "fp32", kind="layer", after=True, bias=True, gates=4, scale=0.9, pad=40)},
        # One token of one sequence through 4-bit weights: two gated projections in one matrix.
        {"name": "linear_i4 1", "op": "linear_i4", "M": 1, "K": 8192, "N": 16384, "group": 128, "zero": False, "dtype": "bf16"},
        # A small serving batch, finely grouped weights with zero points.
        {"name": "linear_i4 13", "op": "linear_i4", "M": 13, "K": 5120, "N": 10240, "group": 32, "zero": True, "dtype": "fp16"},
        # A shard whose sizes are no multiples of a tile or of the group.
        {"name": "linear_i4 odd", "op": "linear_i4", "M": 3, "K": 5001, "N": 1737, "group": 64, "zero": True, "dtype": "bf16"},
        # One token through its four experts.
        {"name": "moe 1", "op": "moe", "T": 1, "K": 5120, "F": 1736, "E": 32, "first": 0, "local": 32, "top_k": 4, "act": "silu", "normalize": True, "dtype": "bf16"},
        # A small serving batch on a rank that holds half of the experts.
        {"name": "moe half 9", "op": "moe", "T": 9, "K": 2048, "F": 1032, "E": 16, "first": 8, "local": 8, "top_k": 2, "act": "gelu", "normalize": False, "dtype": "fp16"},
        # The largest batch of a decoding step: nearly every expert has tokens.
        {"name": "moe 32", "op": "moe", "T": 32, "K": 2048, "F": 1024, "E": 64, "first": 0, "local": 64, "top_k": 8, "act": "silu", "normalize": True, "dtype": "bf16"},
    ]


def draw(rng):
    def size(low, high, odd=0.4):
        n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        if rng.random() >= odd and n >= 64:
            n = n // 16 * 16
        return max(low, min(high, n))

    op = rng.choice(["norm", "norm_grad", "linear_i4", "moe"])
    half = rng.choice(["bf16", "fp16"])
    if op in ("norm", "norm_grad"):
        rows, after = size(1, 16384 if op == "norm" else 8192), rng.random() < 0.4
        gates = rng.choice([0, 0, 1, rows, next(g for g in (7, 5, 4, 3, 2, 1) if rows % g == 0)])
        case = _norm_case(op, rows, size(64, 8192), rng.choice([half, half, "fp32"]), rng.choice(["rms", "rms", "layer"]), True, after,
                          not after or rng.random() < 0.7, rng.random() < 0.3, gates, rng.choice([1.0, 1.0, 0.75]),
                          rng.choice([0.0, 0.0, 1.0]), rng.choice([0, 0, 8, 5]))
        if not after and not gates and rng.random() < 0.2:
            case["residual"], case["scale"] = False, 1.0  # the first block's norm: nothing to add
        while work(case)["bytes"] > 9e8:
            case["rows"] //= 2
            case["gates"] = min(case["gates"], 1)
        return case
    if op == "linear_i4":
        return {"op": op, "M": size(1, 64), "K": size(64, 16384), "N": size(64, 16384), "group": rng.choice([32, 64, 128]), "zero": rng.random() < 0.5, "dtype": half}
    T, K, F = size(1, 64), size(64, 5120), size(64, 2048)
    E = max(2, min(128, int(4e8 / (6 * K * F)), size(2, 128)))
    local = rng.choice([E, E, max(1, E // 2)])
    return {"op": op, "T": T, "K": K, "F": F, "E": E, "first": rng.randrange(E - local + 1), "local": local, "top_k": min(E, rng.choice([1, 2, 4, 6, 8])),
            "act": rng.choice(["silu", "gelu"]), "normalize": rng.random() < 0.6, "dtype": half}


# --------------------------------------------------------------------------------------------------------------- inputs

EPS = 1e-5


def _normal(gen, shape, dtype, scale=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale + mean).to(dtype)


def _prepare_norm(c, s, gen, dtype):
    rows, cols, pad = c["rows"], c["cols"], c["pad"]

    def matrix(scale=1.0, mean=0.0):
        return _normal(gen, (rows, cols + pad), dtype, scale, mean)[:, :cols]

    def vector(mean):
        return _normal(gen, (cols,), dtype, 0.2, mean)

    s["x"] = matrix(0.7, 0.2)
    if c["residual"]:
        s["residual"] = matrix(2.0, -0.3)
    for name, there in (("weight", c["before"]), ("after_weight", c["after"])):
        if there:
            s[name] = vector(1.0 - c["offset"])
            if c["bias"]:
                s[name.replace("weight", "bias")] = vector(0.0)
    if c["gates"]:
        s["gate"] = _normal(gen, (c["gates"], cols), dtype, 0.3, 0.5)
    if c["op"] == "norm_grad":
        # What the forward pass left: the stored r (x itself where nothing was added), and the gradients that come back.
        if c["residual"]:
            s["r"] = _plain_branch(c, s)[0].to(dtype)
            s["dr"] = matrix()
        if c["before"]:
            s["dy"] = matrix()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 6271 + 29)
    c, dtype = case, DTYPES[case["dtype"]]
    s = {"case": case}
    if c["op"] in ("norm", "norm_grad"):
        _prepare_norm(c, s, gen, dtype)
    elif c["op"] == "linear_i4":
        M, K, N, groups = c["M"], c["K"], c["N"], -(-c["K"] // c["group"])
        s["x"] = _normal(gen, (M, K), dtype)
        s["q"] = torch.randint(0, 16, (N, K), generator=gen, device="cuda", dtype=torch.uint8)
        s["scale"] = ((torch.rand((N, groups), generator=gen, device="cuda") + 0.5) / (4.6 * K ** 0.5)).to(dtype)
        if c["zero"]:
            s["zero"] = torch.randint(4, 12, (N, groups), generator=gen, device="cuda", dtype=torch.uint8)
        if own:  # laid out once, as a program does when it loads its weights
            from shot_allreduce_ranks_gb300 import pack_i4
            s["packed"] = pack_i4(s["q"], s["scale"], s.get("zero"), group=c["group"])
    else:
        T, K, F, n = c["T"], c["K"], c["F"], c["local"]
        s["x"] = _normal(gen, (T, K), dtype)
        # Logits in 16 bits, as a router in the model's type gives them: some are equal.
        s["logits"] = _normal(gen, (T, c["E"]), dtype, 1.5)
        s["w_gate"] = _normal(gen, (n, F, K), dtype, K ** -0.5)
        s["w_up"] = _normal(gen, (n, F, K), dtype, K ** -0.5)
        s["w_down"] = _normal(gen, (n, K, F), dtype, F ** -0.5)
    return s


# ------------------------------------------------------------------------------------------------------------------ run

def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case["op"], case, state)


def _run_own(op, c, s):
    import shot_allreduce_ranks_gb300 as ar

    if op == "linear_i4":
        return ar.linear_i4(s["x"], s["packed"])
    if op == "moe":
        return ar.moe_ffn(s["x"], s["logits"], s["w_gate"], s["w_up"], s["w_down"], c["top_k"], activation=c["act"],
                          normalize=c["normalize"], first_expert=c["first"], routing=True)
    if op == "norm":
        return ar.residual_norm(s["x"], s.get("residual"), s.get("weight"), s.get("bias"), s.get("after_weight"), s.get("after_bias"),
                                s.get("gate"), kind=c["kind"], eps=EPS, residual_scale=c["scale"], weight_offset=c["offset"])
    return ar.residual_norm_backward(s.get("dy"), s.get("dr"), s["x"], s.get("r"), s.get("weight"), s.get("bias"), s.get("after_weight"),
                                     s.get("after_bias"), s.get("gate"), kind=c["kind"], eps=EPS, residual_scale=c["scale"],
                                     weight_offset=c["offset"])


def _hat(v, kind):
    """(the normalised rows, the factor they were multiplied by)"""
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    f = 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    return v * f, f


def _plain_branch(c, s):
    """(r before rounding, the branch before its gate, the gate for every row)"""
    z = s["x"].float()
    if c["after"]:
        z = _hat(z, c["kind"])[0] * (s["after_weight"].float() + c["offset"])
        z = z + s["after_bias"].float() if c["bias"] else z
    gate = s["gate"].float().repeat_interleave(c["rows"] // c["gates"], dim=0) if c["gates"] else None
    r = z if gate is None else gate * z
    if c["residual"]:
        r = r + c["scale"] * s["residual"].float()
    return r, z, gate


def _hat_grad(dhat, hat, f, kind):
    """The gradient of the rows from that of the normalised rows."""
    d = dhat - hat * (dhat * hat).mean(dim=1, keepdim=True)
    return f * (d - dhat.mean(dim=1, keepdim=True) if kind == "layer" else d)


def _plain_norm(c, s, dtype):
    r = _plain_branch(c, s)[0]
    y = None
    if c["before"]:
        y = _hat(r, c["kind"])[0] * (s["weight"].float() + c["offset"])
        y = (y + s["bias"].float() if c["bias"] else y).to(dtype)
    return (r.to(dtype) if c["residual"] else None), y


def _plain_norm_grad(c, s, dtype):
    out = dict.fromkeys(("dx", "dresidual", "dweight", "dbias", "dafter_weight", "dafter_bias", "dgate"))
    g = s["dr"].float() if c["residual"] else 0.0
    if c["before"]:
        dy = s["dy"].float()
        hat, f = _hat((s["r"] if c["residual"] else s["x"]).float(), c["kind"])
        out["dweight"] = (dy * hat).sum(dim=0)
        out["dbias"] = dy.sum(dim=0) if c["bias"] else None
        g = g + _hat_grad(dy * (s["weight"].float() + c["offset"]), hat, f, c["kind"])
    out["dresidual"] = c["scale"] * g if c["residual"] else None
    _, z, gate = _plain_branch(c, s)
    if c["gates"]:
        out["dgate"] = (g * z).reshape(c["gates"], -1, c["cols"]).sum(dim=1)
        g = g * gate
    if c["after"]:
        hat, f = _hat(s["x"].float(), c["kind"])
        out["dafter_weight"] = (g * hat).sum(dim=0)
        out["dafter_bias"] = g.sum(dim=0) if c["bias"] else None
        g = _hat_grad(g * (s["after_weight"].float() + c["offset"]), hat, f, c["kind"])
    out["dx"] = g
    return tuple(None if v is None else v.to(dtype) for v in out.values())


GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def _plain_moe(c, s, dtype):
    T, k, n = c["T"], c["top_k"], c["local"]
    logits = s["logits"].float()
    value, expert = torch.sort(logits, dim=1, descending=True, stable=True)  # equal logits: the lowest index first
    value, expert = value[:, :k], expert[:, :k]
    share = torch.exp(value - value[:, :1])
    share = share / (share if c["normalize"] else torch.exp(logits - value[:, :1])).sum(dim=1, keepdim=True)
    here = (expert >= c["first"]) & (expert < c["first"] + n)
    # The experts that are computed, for all tokens: one for each token and choice, or every one where those are fewer.
    mine = torch.where(here, expert - c["first"], 0).reshape(-1)
    coefficient = torch.where(here, share, 0.0).reshape(-1)
    token = torch.arange(T, device=logits.device).repeat_interleave(k)
    if T * k <= n:
        slots = mine
        c_tp = torch.zeros((T, T * k), device=logits.device)
        c_tp[token, torch.arange(T * k, device=logits.device)] = coefficient
    else:
        slots = torch.arange(n, device=logits.device)
        c_tp = torch.zeros((T, n), device=logits.device).index_put((token, mine), coefficient, accumulate=True)
    x = s["x"].float()[None].expand(len(slots), -1, -1)
    g = torch.bmm(x, s["w_gate"][slots].float().transpose(1, 2))
    if c["act"] == "silu":
        g = g / (1.0 + torch.exp(-g))
    else:
        g = 0.5 * g * (1.0 + torch.tanh(GELU_C * (g + GELU_A * g * g * g)))
    h = g * torch.bmm(x, s["w_up"][slots].float().transpose(1, 2)) * c_tp.T[:, :, None]
    y = torch.bmm(h, s["w_down"][slots].float().transpose(1, 2)).sum(dim=0)
    return y.to(dtype), expert.to(torch.int32), share


def _run_plain(op, c, s):
    dtype = DTYPES[c["dtype"]]
    if op == "norm":
        return _plain_norm(c, s, dtype)
    if op == "norm_grad":
        return _plain_norm_grad(c, s, dtype)
    if op == "moe":
        return _plain_moe(c, s, dtype)
    spread = lambda t: t.float().repeat_interleave(c["group"], dim=1)[:, :c["K"]]  # noqa: E731
    w = (s["q"].float() - (spread(s["zero"]) if c["zero"] else 8.0)) * spread(s["scale"])
    return (s["x"].float() @ w.T).to(dtype)


# -------------------------------------------------------------------------------------------------- the values in 64 bits

def _exact_rows(v, weight, bias, c):
    """The norm of the definition: rows less their mean (layer), over the root of their mean square, times the weight."""
    if weight is None:
        return v
    if c["kind"] == "layer":
        v = v - v.sum(1, keepdim=True) / v.shape[1]
    v = v * torch.rsqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS) * (c["offset"] + weight)
    return v if bias is None else v + bias


def _exact_norm(c, s, d):
    names = ("x", "residual", "weight", "bias", "after_weight", "after_bias", "gate")
    p = {k: d[k].requires_grad_(c["op"] == "norm_grad") if k in d else None for k in names}
    branch = _exact_rows(p["x"], p["after_weight"], p["after_bias"], c)
    if c["gates"]:
        branch = (branch.reshape(c["gates"], -1, c["cols"]) * p["gate"][:, None, :]).reshape(c["rows"], c["cols"])
    r = branch + c["scale"] * p["residual"] if c["residual"] else branch
    if c["op"] == "norm":
        return (r if c["residual"] else None), (_exact_rows(r, p["weight"], p["bias"], c) if c["before"] else None)
    # The backward pass starts from the stored r, which was rounded: its norm is differentiated there.
    back = d["dr"] if c["residual"] else torch.zeros_like(r)
    if c["before"]:
        at = (d["r"] if c["residual"] else d["x"]).detach().clone().requires_grad_()
        _exact_rows(at, p["weight"], p["bias"], c).backward(d["dy"])
        back = back + at.grad
    r.backward(back)
    order = ("x", "residual", "weight", "bias", "after_weight", "after_bias", "gate")
    return tuple(None if p[k] is None else p[k].grad for k in order)


def _exact_moe(c, s, d):
    z = d["logits"].cpu()
    y = torch.zeros_like(d["x"])
    share, order = [], []
    for t in range(c["T"]):
        best = sorted(range(c["E"]), key=lambda e: (-float(z[t, e]), e))[:c["top_k"]]
        p = torch.softmax(z[t], 0)[best]
        order.append(best)
        share.append(p / p.sum() if c["normalize"] else p)
    for e in range(c["local"]):
        rows = [(t, i) for t in range(c["T"]) for i, b in enumerate(order[t]) if b == c["first"] + e]
        if not rows:
            continue
        at = [t for t, _ in rows]
        x = d["x"][at]
        g = torch.mm(x, s["w_gate"][e].double().t())
        f = torch.nn.functional.silu(g) if c["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        h = f * torch.mm(x, s["w_up"][e].double().t())
        part = torch.mm(h, s["w_down"][e].double().t())
        y[at] += part * torch.stack([share[t][i] for t, i in rows]).to(part.device)[:, None]
    return y, None, torch.stack(share).to(y.device)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("w_gate", "w_up", "w_down", "q")}
    if c["op"] in ("norm", "norm_grad"):
        return _exact_norm(c, s, d)
    if c["op"] == "moe":
        return _exact_moe(c, s, d)
    y = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device="cuda")
    for j in range(0, c["K"], c["group"]):
        q = s["q"][:, j:j + c["group"]].double()
        at = j // c["group"]
        q = q - (d["zero"][:, at:at + 1] if c["zero"] else 8.0)
        y += torch.mm(d["x"][:, j:j + c["group"]], q.t()) * d["scale"][:, at][None, :]
    return y


# ----------------------------------------------------------------------------------------------------------------- work

def work(case):
    c, e = case, 4 if case["dtype"] == "fp32" else 2
    if c["op"] in ("norm", "norm_grad"):
        n = c["rows"] * c["cols"]
        vectors = (c["before"] + c["after"]) * (1 + c["bias"]) + c["gates"]
        if c["op"] == "norm":
            # x and the residual are read, r and y written.
            streams = 1 + 2 * c["residual"] + c["before"]
            return {"bytes": e * (n * streams + vectors * c["cols"]), "flops": 8 * n}
        # dy, dr, r and (for a gate or the norm after the block) x are read, dx written; the residual's gradient is dx where
        # neither a gate, a norm nor a scale stands between them.
        branch = bool(c["after"] or c["gates"])
        streams = c["before"] + c["residual"] + (c["before"] if c["residual"] else 1) + branch + 1 + (c["residual"] and (branch or c["scale"] != 1.0))
        return {"bytes": e * (n * streams + 2 * vectors * c["cols"]), "flops": 14 * n}
    if c["op"] == "linear_i4":
        M, K, N = c["M"], c["K"], c["N"]
        groups = -(-K // c["group"])
        return {"bytes": N * K / 2 + N * groups * (2.5 if c["zero"] else 2) + 2 * M * (K + N), "flops": 2 * M * K * N}
    T, K, F, E, k, n = (c[key] for key in ("T", "K", "F", "E", "top_k", "local"))
    # The experts that a batch of random tokens is sent to, on the mean.
    used = n * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": used * 6 * K * F + 4 * T * K + 2 * T * E + 8 * T * k, "flops": 6 * T * k * n / E * K * F}
