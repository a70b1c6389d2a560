"""The operators around the expert block, case by case: expert routing, the norm in front of the
block, and 8-bit activation checkpoints.

Each case is one pass through an operator as a training step or a serving step calls it.
`run` computes it in the plain form (elementary torch operations, 32 bits, and 64 bits for the
keys that routing decisions compare), or, with `own` set, through the library's entry points.

Routing.  Logits l [T,E] in fp32; a logit (or a bias) that is NaN, -inf or the lowest finite
value masks its expert.  Scores s = softmax(l) or sigmoid(l); selection key s + b with a balance
bias b [E] and the order of l without one.  With groups, a group's score is the sum of its
`group_best` largest keys, and only experts of the `top_groups` best groups are eligible.  The k
largest keys are selected, largest first, ties to the lower index; their weights are
scale * s_j, divided by the selected scores' sum with `renormalize`.

Norm.  n = (x - mean) / sqrt(var + eps) * g + b per row ("layer"), or x / sqrt(mean(x^2) + eps)
* g ("rms").  With a residual, x_out = x + y (rounded once) is what is normalised.

Checkpoint.  Blocks of 32 features share a power-of-two scale 2^S; elements are E4M3 values
(S the smallest integer with max|x| <= 448 * 2^S) or 8-bit integers (max|x| <= 127 * 2^S).
"""

import math

import torch

own = False

LOWEST = torch.finfo(torch.float32).min
EPS = 1e-5


def listed():
    return [
        # one new token of a 32-expert layer, softmax over the selected: latency alone
        {"name": "route 1 token, 32 experts", "op": "route", "T": 1, "E": 32, "k": 4,
         "scores": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_best": 1,
         "renormalize": True, "scale": 1.0, "backward": False},
        # a serving batch of single tokens of a wide layer: groups, balance bias
        {"name": "route 64 tokens, 256 experts", "op": "route", "T": 64, "E": 256, "k": 8,
         "scores": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2,
         "renormalize": True, "scale": 2.5, "backward": False},
        # a training step's routing over 128 experts with the scores as weights: the softmax's
        # dense gradient
        {"name": "route 16384 tokens, softmax", "op": "route", "T": 16384, "E": 128, "k": 4,
         "scores": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_best": 1,
         "renormalize": False, "scale": 1.0, "backward": True},
        # a training step over 256 experts: sigmoid, balance bias, 4 of 8 groups
        {"name": "route 32768 tokens, groups", "op": "route", "T": 32768, "E": 256, "k": 8,
         "scores": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2,
         "renormalize": True, "scale": 2.5, "backward": True},
        # the norm in front of the block for one new token
        {"name": "norm 1 token", "op": "norm", "T": 1, "H": 2880, "kind": "rms",
         "dtype": "bf16", "params": "bf16", "residual": True, "backward": False},
        # one layer's training step, residual add in front, weights' gradient behind
        {"name": "norm 8192 tokens", "op": "norm", "T": 8192, "H": 2880, "kind": "layer",
         "dtype": "bf16", "params": "bf16", "residual": True, "backward": True},
        # odd sizes: rows that no vector width divides, fp32 stream
        {"name": "norm 1237 tokens, odd", "op": "norm", "T": 1237, "H": 1001, "kind": "layer",
         "dtype": "fp32", "params": "fp32", "residual": False, "backward": True},
        # a long sequence's rms norm, forward and backward
        {"name": "norm 32768 tokens", "op": "norm", "T": 32768, "H": 2880, "kind": "rms",
         "dtype": "bf16", "params": "fp32", "residual": False, "backward": True},
        # the tiny block's rows stored and read back
        {"name": "checkpoint 64 tokens", "op": "checkpoint", "T": 64, "H": 256, "format": "e4m3",
         "dtype": "bf16", "use": "store"},
        # one layer's input stored as 8-bit integers and read back
        {"name": "checkpoint 16384 tokens", "op": "checkpoint", "T": 16384, "H": 2880,
         "format": "int8", "dtype": "bf16", "use": "store"},
        # a ragged batch: forward with the checkpoint, then the recompute and the backward from it
        {"name": "checkpoint 1000 tokens, norm", "op": "checkpoint", "T": 1000, "H": 1056,
         "format": "int8", "dtype": "bf16", "use": "norm"},
        # one block boundary of the 24-block stack, forward and backward
        {"name": "checkpoint 32768 tokens, norm", "op": "checkpoint", "T": 32768, "H": 2880,
         "format": "e4m3", "dtype": "bf16", "use": "norm"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "norm", "checkpoint"])
    if op == "route":
        E = rng.choice([_spread(rng, 2, 256), 32, 64, 128, 160, 256])
        divisors = [g for g in range(1, 33) if E % g == 0]
        groups = rng.choice(divisors) if rng.random() < 0.5 else 1
        top_groups = rng.randint(1, groups)
        size = E // groups
        return {"op": op, "T": _spread(rng, 1, 32768), "E": E,
                "k": rng.randint(1, min(8, top_groups * size)),
                "scores": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": groups, "top_groups": top_groups,
                "group_best": rng.choice([1, 2]) if size > 1 else 1,
                "renormalize": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]),
                "backward": rng.random() < 0.6}
    if op == "norm":
        H = rng.choice([_spread(rng, 32, 8192), 32 * _spread(rng, 1, 256)])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = 32768 * 2880 // (H * (1 if dtype == "bf16" else 2))
        return {"op": op, "T": _spread(rng, 1, min(32768, most)), "H": H,
                "kind": rng.choice(["layer", "rms"]), "dtype": dtype,
                "params": rng.choice(["bf16", "fp32"]), "residual": rng.random() < 0.5,
                "backward": rng.random() < 0.6}
    H = 32 * _spread(rng, 1, 256)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    most = 32768 * 2880 // (H * (1 if dtype == "bf16" else 2))
    return {"op": op, "T": _spread(rng, 1, min(32768, most)), "H": H,
            "format": rng.choice(["e4m3", "int8"]), "dtype": dtype,
            "use": rng.choice(["store", "norm"])}


# ---- inputs ------------------------------------------------------------------------------
def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _rows(g, T, H, dtype, wide=False):
    """Rows of a residual stream: normal features, and with `wide` a few channels far larger."""
    x = torch.randn(T, H, generator=g, device="cuda")
    if wide:
        gain = torch.rand(H, generator=g, device="cuda")
        x *= torch.where(gain > 0.99, 30.0, 1.0) * 2.0
        x += 0.25
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        logits = torch.randn(T, E, generator=g, device="cuda") * 1.5
        # the gradient of the loss with respect to the routing weights
        state = {"case": case, "logits": logits,
                 "d_w": torch.randn(T, k, generator=g, device="cuda")}
        state["bias"] = (torch.randn(E, generator=g, device="cuda") * 0.05
                         if case["bias"] else None)
        return state
    H, dtype = case["H"], _dtype(case["dtype"])
    state = {"case": case, "x": _rows(g, T, H, dtype, wide=True)}
    if case["op"] == "norm" or case["use"] == "norm":
        params = _dtype(case.get("params", "bf16"))
        state["weight"] = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(params)
        state["bias"] = None
        if case.get("kind", "layer") == "layer":
            state["bias"] = (0.1 * torch.randn(H, generator=g, device="cuda")).to(params)
        state["y"] = _rows(g, T, H, dtype) if case.get("residual", True) else None
        if case.get("backward", True):
            state["d_out"] = _rows(g, T, H, dtype)
            # the gradient that reaches the rows past the norm, through the residual stream
            state["g"] = _rows(g, T, H, dtype) if case.get("residual", True) else None
    return state


# ---- one pass ----------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if case["op"] == "route":
        return _run_route(state)
    if case["op"] == "norm":
        return _run_norm(state)
    return _run_store(state) if case["use"] == "store" else _run_checkpointed_norm(state)


def _run_route(state):
    case, logits, bias = state["case"], state["logits"], state["bias"]
    if own:
        from mxfp4_quantized_moe_b200 import moe
        r = moe.Routing(k=case["k"], scores=case["scores"], groups=case["groups"],
                        top_groups=case["top_groups"], group_best=case["group_best"],
                        renormalize=case["renormalize"], scale=case["scale"])
        idx, w = moe.route(r, logits, bias)
        if not case["backward"]:
            return idx, w
        return idx, w, moe.route_backward(r, logits, idx, w, state["d_w"])
    idx, w = _plain_route(case, logits, bias)
    if not case["backward"]:
        return idx, w
    return idx, w, _plain_route_backward(case, logits, idx, w, state["d_w"])


def _run_norm(state):
    case, x, y = state["case"], state["x"], state["y"]
    weight, bias, kind = state["weight"], state["bias"], case["kind"]
    if own:
        from mxfp4_quantized_moe_b200 import moe
        f = moe.norm_forward(x, weight, bias, kind=kind, eps=EPS, y=y)
        rows = x if y is None else f.x_out
        out = {"out": f.out} if y is None else {"out": f.out, "x_out": f.x_out}
        if case["backward"]:
            out["dx"], out["d_weight"], d_bias = moe.norm_backward(
                state["d_out"], rows, f.mean, f.rstd, weight, kind=kind, g=state["g"])
            if kind == "layer":
                out["d_bias"] = d_bias
        return out
    rows = x if y is None else x + y
    n, mean, rstd = _plain_norm(rows.float(), weight, bias, kind)
    out = {"out": n.to(x.dtype)} if y is None else {"out": n.to(x.dtype), "x_out": rows}
    if case["backward"]:
        out.update(_plain_norm_backward(state["d_out"], rows.float(), mean, rstd, weight, kind,
                                        state["g"]))
    return out


def _run_store(state):
    case, x = state["case"], state["x"]
    if own:
        from mxfp4_quantized_moe_b200 import moe
        return moe.checkpoint_unpack(moe.checkpoint_pack(x, case["format"]), x.dtype)
    return _plain_read(*_plain_store(x, case["format"])).to(x.dtype)


def _run_checkpointed_norm(state):
    """The forward at a block boundary (residual add, checkpoint, norm), then the backward: the
    norm again from the checkpoint, and its gradients."""
    case, x, y = state["case"], state["x"], state["y"]
    weight, bias, d_out, g = state["weight"], state["bias"], state["d_out"], state["g"]
    if own:
        from mxfp4_quantized_moe_b200 import moe
        f = moe.norm_forward(x, weight, bias, kind="layer", eps=EPS, y=y,
                             checkpoint=case["format"])
        again = moe.norm_forward(f.checkpoint, weight, bias, kind="layer", eps=EPS,
                                 dtype=x.dtype)
        dx, d_weight, d_bias = moe.norm_backward(d_out, f.checkpoint, again.mean, again.rstd,
                                                 weight, kind="layer", g=g)
        return {"x_out": f.x_out, "out": f.out, "again": again.out, "dx": dx,
                "d_weight": d_weight, "d_bias": d_bias}
    rows = x + y
    n, _, _ = _plain_norm(rows.float(), weight, bias, "layer")
    stored = _plain_read(*_plain_store(rows, case["format"]))
    again, mean, rstd = _plain_norm(stored, weight, bias, "layer")
    out = {"x_out": rows, "out": n.to(x.dtype), "again": again.to(x.dtype)}
    out.update(_plain_norm_backward(d_out, stored, mean, rstd, weight, "layer", g))
    return out


# ---- plain forms -------------------------------------------------------------------------
def _absent(v):
    return ~(v > LOWEST)  # NaN, -inf and the lowest finite value


def _plain_scores(case, logits):
    """Scores in 64 bits: routing decisions compare them next to one another."""
    gone = _absent(logits)
    l = logits.double().clamp(max=-LOWEST)
    if case["scores"] == "sigmoid":
        return torch.where(gone, 0.0, 1.0 / (1.0 + torch.exp(-l)))
    l = torch.where(gone, -math.inf, l)
    top = l.max(dim=1, keepdim=True).values
    z = torch.where(gone, 0.0, torch.exp(l - torch.where(top > -math.inf, top, 0.0)))
    total = z.sum(dim=1, keepdim=True)
    return z / torch.where(total > 0, total, 1.0)


def _plain_route(case, logits, bias):
    T, E = logits.shape
    groups, k = case["groups"], case["k"]
    s = _plain_scores(case, logits)
    gone = _absent(logits)
    if bias is not None:
        gone = gone | _absent(bias)
        key = s + bias.double().clamp(max=-LOWEST)
    else:
        key = logits.double().clamp(max=-LOWEST)
    if groups > 1:
        score = torch.where(gone, -math.inf, key if bias is not None else s)
        best = score.view(T, groups, E // groups).sort(dim=2, descending=True).values
        best = best[:, :, :case["group_best"]]
        some = best[:, :, 0] > -math.inf
        total = torch.where(best > -math.inf, best, 0.0).sum(dim=2)
        order = torch.where(some, total, -math.inf).sort(dim=1, descending=True, stable=True)
        kept = torch.zeros(T, groups, dtype=torch.bool, device=logits.device)
        kept.scatter_(1, order.indices[:, :case["top_groups"]], True)
        out = ~kept.repeat_interleave(E // groups, dim=1)
    else:
        out = torch.zeros_like(gone)
    # eligible experts first, then the masked ones of the kept groups, then the others
    key = torch.where(gone, -1e300, key)
    key = torch.where(out, -math.inf, key)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    sel = torch.where(gone.gather(1, idx), 0.0, s.gather(1, idx))
    if case["renormalize"]:
        total = sel.sum(dim=1, keepdim=True)
        sel = sel / torch.where(total > 0, total, 1.0)
    return idx.int(), (case["scale"] * sel).float()


def _plain_route_backward(case, logits, idx, w, d_w):
    idx, scale = idx.long(), case["scale"]
    s = _plain_scores(case, logits).float()
    if case["renormalize"]:
        d_log = w * (d_w - (w * d_w).sum(dim=1, keepdim=True) / scale)
    else:
        d_log = w * d_w
    d = torch.zeros_like(logits)
    if case["scores"] == "sigmoid":
        rest = 1.0 / (1.0 + torch.exp(logits.gather(1, idx)))  # 1 - sigmoid
        return d.scatter_add_(1, idx, torch.where(w != 0, d_log * rest, 0.0))
    d.scatter_add_(1, idx, d_log)
    return d if case["renormalize"] else d - s * d_log.sum(dim=1, keepdim=True)


def _plain_norm(rows, weight, bias, kind):
    mean = rows.mean(dim=1) if kind == "layer" else torch.zeros_like(rows[:, 0])
    away = rows - mean[:, None]
    rstd = 1.0 / torch.sqrt((away * away).mean(dim=1) + EPS)
    n = away * rstd[:, None] * weight.float()
    return n if bias is None else n + bias.float(), mean, rstd


def _plain_norm_backward(d_out, rows, mean, rstd, weight, kind, g):
    d = d_out.float()
    hat = (rows - mean[:, None]) * rstd[:, None]
    part = d * weight.float()
    dx = part - hat * (part * hat).mean(dim=1, keepdim=True)
    if kind == "layer":
        dx = dx - part.mean(dim=1, keepdim=True)
    dx = dx * rstd[:, None]
    if g is not None:
        dx = dx + g.float()
    out = {"dx": dx.to(d_out.dtype), "d_weight": (d * hat).sum(dim=0)}
    if kind == "layer":
        out["d_bias"] = d.sum(dim=0)
    return out


def _two_to(S):
    """2^S in fp32, exactly, for whole S within [-126, 127] (S an int32 tensor)."""
    return ((S + 127) << 23).view(torch.float32)


def _plain_store(rows, format):
    """The elements as values in units of 2^S, and S, by blocks of 32."""
    b = rows.float().view(rows.shape[0], -1, 32)
    most = b.abs().amax(dim=2, keepdim=True)
    m, e = torch.frexp(most)  # most = m * 2^e, m in [0.5, 1)
    if format == "e4m3":
        S = torch.where(m > 0.875, e - 8, e - 9)  # 448 = 0.875 * 2^9
        S = torch.where(most > 0, S, -126).clamp(-126, 120)
        v = (b * _two_to(-S)).to(torch.float8_e4m3fn).float()
        v = torch.where(S == 120, v.clamp(-240.0, 240.0), v)  # stays finite times 2^120
    else:
        S = torch.where(m > 127 / 128, e - 6, e - 7)  # 127 = 127/128 * 2^7
        S = torch.where(most > 0, S, -126).clamp(-126, 121)
        v = (b * _two_to(-S)).round().clamp(-127.0, 127.0)
    return v, S


def _plain_read(v, S):
    return (v * _two_to(S)).view(v.shape[0], -1)


# ---- work --------------------------------------------------------------------------------
def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        n = 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0)
        flops = 4 * T * E
        if case["backward"]:
            # the weights' gradient in, the logits' out; the logits, indices and weights are
            # read again
            n += 4 * T * k + 4 * T * E + 8 * T * k
            dense = case["scores"] == "softmax" and not case["renormalize"]
            n += 4 * T * E if dense else (4 * T * k if case["scores"] == "sigmoid" else 0)
            flops += 2 * T * E
        return {"bytes": n, "flops": flops}
    H, size = case["H"], 2 if case["dtype"] == "bf16" else 4
    cells, packed = T * H, 1 + 1 / 32
    if case["op"] == "checkpoint" and case["use"] == "store":
        return {"bytes": cells * (2 * size + 2 * packed), "flops": 4 * cells}
    params = 2 if case.get("params", "bf16") == "bf16" else 4
    # rows [and the residual] in, n [and the sum] out
    n = cells * size * (4 if case.get("residual", True) else 2) + 2 * H * params
    flops = 8 * cells
    back = case.get("backward", True)
    if case["op"] == "checkpoint":
        n += cells * packed                              # the checkpoint out
        n += cells * (packed + size)                     # in again, n out again
        n += cells * (packed + 3 * size) + 8 * H         # in again, d_out, g in, dx out
        flops += 20 * cells
    elif back:
        n += cells * size * (4 if case["residual"] else 3) + 8 * H
        flops += 12 * cells
    return {"bytes": n, "flops": flops}


# ---- the definition in 64 bits -----------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, state)
    if case["op"] == "checkpoint" and case["use"] == "store":
        return _exact_stored(state["x"].double(), case["format"])
    return _exact_norm(case, state)


def _exact_route(case, state):
    """One token's selection by repeated search for the largest key, all tokens at once."""
    l = state["logits"].double()
    T, E = l.shape
    rows = torch.arange(T, device=l.device)
    if case["scores"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.softmax(l, dim=1)
    key = l if state["bias"] is None else s + state["bias"].double()
    free = torch.ones(T, E, dtype=torch.bool, device=l.device)
    if case["groups"] > 1:
        of = torch.arange(E, device=l.device) // (E // case["groups"])
        by = s if state["bias"] is None else key
        total = []
        for grp in range(case["groups"]):
            mine = by[:, of == grp]
            total.append(mine.topk(case["group_best"], dim=1).values.sum(dim=1))
        total = torch.stack(total, dim=1)
        free &= False
        for _ in range(case["top_groups"]):
            grp = total.argmax(dim=1)
            free |= of[None, :] == grp[:, None]
            total[rows, grp] = -math.inf
    key = torch.where(free, key, -math.inf)
    idx, sel = [], []
    for _ in range(case["k"]):
        e = key.argmax(dim=1)
        idx.append(e)
        sel.append(s[rows, e])
        key[rows, e] = -math.inf
    idx, sel = torch.stack(idx, dim=1), torch.stack(sel, dim=1)
    c, dw = case["scale"], state["d_w"].double()
    total = sel.sum(dim=1, keepdim=True)
    w = c * sel / total if case["renormalize"] else c * sel
    if not case["backward"]:
        return None, w
    if case["renormalize"]:  # d w_i / d s_j = c (delta_ij - w_i / c) / total
        d_s = c / total * (dw - (dw * w).sum(dim=1, keepdim=True) / c)
    else:
        d_s = c * dw
    full = torch.zeros_like(s)
    for j in range(case["k"]):
        full[rows, idx[:, j]] += d_s[:, j]
    if case["scores"] == "sigmoid":
        return None, w, full * s * (1.0 - s)
    return None, w, s * (full - (full * s).sum(dim=1, keepdim=True))


def _bits_of_power(n):
    """2^n in 64 bits from its exponent field (a power function need not be exact)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_stored(x, format):
    """Each value rounded to the nearest element of its block's grid, ties to even."""
    b = x.reshape(x.shape[0], x.shape[1] // 32, 32)
    most = b.abs().amax(dim=2, keepdim=True)
    limit = 448.0 if format == "e4m3" else 127.0
    S = torch.ceil(torch.log2(torch.where(most > 0, most, 1.0) / limit))
    unit = _bits_of_power(S)
    unit = torch.where(most > limit * unit, unit * 2, unit)      # log2 next to a whole number
    unit = torch.where(most <= limit * unit / 2, unit / 2, unit)
    v = b / unit
    if format == "e4m3":
        lead = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
        step = _bits_of_power(lead - 3)
    else:
        step = 1.0
    return (torch.round(v / step) * step * unit).reshape(x.shape)


def _exact_norm(case, state):
    stored = case["op"] == "checkpoint"
    layer = case.get("kind", "layer") == "layer"
    x, H = state["x"], case["H"]
    out = {}
    if state["y"] is not None:
        x = (x.double() + state["y"].double()).to(x.dtype)  # what the stream holds
        out["x_out"] = state["x"].double() + state["y"].double()
    w, b = state["weight"].double(), state["bias"]

    def normed(v):
        if layer:
            v = v - v.sum(dim=1, keepdim=True) / H
        r = ((v * v).sum(dim=1, keepdim=True) / H + EPS) ** -0.5
        return v * r, r

    def scaled(hat):
        return hat * w if b is None else hat * w + b.double()

    hat, r = normed(x.double())
    out["out"] = scaled(hat)
    if stored:
        hat, r = normed(_exact_stored(x.double(), case["format"]))
        out["again"] = scaled(hat)
    if case.get("backward", True):
        d = state["d_out"].double()
        out["d_weight"] = torch.einsum("th,th->h", d, hat)
        if layer:
            out["d_bias"] = torch.einsum("th->h", d)
        a = d * w
        dx = a - hat * torch.einsum("th,th->t", a, hat)[:, None] / H
        if layer:
            dx -= torch.einsum("th->t", a)[:, None] / H
        dx *= r
        out["dx"] = dx if state["g"] is None else dx + state["g"].double()
    return out
