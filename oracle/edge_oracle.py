"""Plain fp64 CPU restatement of the operators at the expert block's edge: expert routing with
scores, balance bias and groups, the layer / rms norm, and 8-bit activation checkpoints.

TEST INFRASTRUCTURE ONLY, like the block's oracle: slow on purpose, a loop over tokens where a
decision is taken, and no code shared with the CUDA path.
"""

from __future__ import annotations

import numpy as np

from .mxfp4_oracle import round_e4m3

LOWEST = float(np.finfo(np.float32).min)


def _masked(v):
    return not v > LOWEST  # NaN, -inf, the lowest finite value


def _scores(row, scores):
    """fp64 scores of one token's logits; masked logits score 0, +inf is the largest value."""
    gone = np.array([_masked(v) for v in row])
    l = np.where(gone, 0.0, np.minimum(row, -LOWEST))
    with np.errstate(over="ignore"):
        if scores == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        elif gone.all():
            s = np.zeros(len(row))
        else:
            z = np.where(gone, 0.0, np.exp(l - l[~gone].max()))
            s = z / z.sum()
    return np.where(gone, 0.0, s), gone


def _log_scores(l, scores):
    """log s up to a constant per token, from unmasked logits (no underflow)."""
    return -np.logaddexp(0.0, -l) if scores == "sigmoid" else l


def route(logits, k, bias=None, scores="softmax", groups=1, top_groups=1, group_best=1,
          renormalize=True, scale=1.0):
    """(idx int64 [T,k], w fp64 [T,k]) by the definition, one token and one choice at a time."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    idx = np.zeros((T, k), dtype=np.int64)
    w = np.zeros((T, k))
    size = E // groups
    for t in range(T):
        s, gone = _scores(logits[t], scores)
        if bias is not None:
            b = np.asarray(bias, dtype=np.float64)
            gone = gone | np.array([_masked(v) for v in b])
            key = s + np.minimum(np.where(gone, 0.0, b), -LOWEST)
        else:
            key = np.minimum(np.where(gone, 0.0, logits[t]), -LOWEST)
        eligible = np.ones(E, dtype=bool)
        if groups > 1:
            # the largest score is the largest logit's, which fp64 scores may no longer tell
            by = key if bias is not None or group_best == 1 else s
            total = []
            for g in range(groups):
                mine = sorted((by[e] for e in range(g * size, (g + 1) * size) if not gone[e]),
                              reverse=True)
                total.append(sum(mine[:group_best]) if mine else -np.inf)
            best = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
            eligible = np.isin(np.arange(E) // size, best)
        order = sorted((e for e in range(E) if eligible[e]),
                       key=lambda e: (bool(gone[e]), 0.0 if gone[e] else -key[e], e))
        idx[t] = order[:k]
        live = [e for e in idx[t] if not gone[e]]
        if live:
            if renormalize:
                a = _log_scores(np.minimum(logits[t][live], -LOWEST), scores)
                p = np.exp(a - a.max())
                p = p / p.sum()
            else:
                p = s[live]
            w[t, :len(live)] = scale * p  # masked experts come last
    return idx, w


def route_backward(logits, idx, w, d_w, scores="softmax", renormalize=True, scale=1.0):
    """d_logits [T,E]: the Jacobian of w with respect to every logit, applied to d_w."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    d = np.zeros((T, E))
    for t in range(T):
        s, _ = _scores(logits[t], scores)
        for j, e in enumerate(idx[t]):
            if w[t, j] == 0.0 or not 0 <= e < E:
                continue
            # dw_j/dl_m: w_j times the derivative of log w_j
            dlog = np.zeros(E)
            dlog[e] += 1.0 - s[e] if scores == "sigmoid" else 1.0
            if renormalize:
                for i, f in enumerate(idx[t]):
                    if 0 <= f < E:
                        p = w[t, i] / scale
                        dlog[f] -= p * (1.0 - s[f]) if scores == "sigmoid" else p
            elif scores == "softmax":
                dlog -= s
            d[t] += d_w[t, j] * w[t, j] * dlog
    return d


def norm(x, weight=None, bias=None, kind="layer", eps=1e-5):
    """(out, mean, rstd) of the rows of x in fp64."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if kind == "layer" else np.zeros(len(x))
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    out = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        out = out * weight
    if bias is not None:
        out = out + bias
    return out, mean, rstd


def norm_backward(d_out, x, weight=None, kind="layer", eps=1e-5, g=None):
    """(dx [+ g], d_weight, d_bias) in fp64."""
    d_out, x = np.asarray(d_out, np.float64), np.asarray(x, np.float64)
    xh, _, rstd = norm(x, kind=kind, eps=eps)
    v = d_out if weight is None else d_out * weight
    dx = v - xh * (v * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - v.mean(axis=1, keepdims=True)
    dx = dx * rstd[:, None]
    return dx if g is None else dx + g, (d_out * xh).sum(axis=0), d_out.sum(axis=0)


def checkpoint(x, format):
    """(codes uint8, scales uint8, values fp64) of rows x [T,H], block by block of 32."""
    x = np.asarray(x, dtype=np.float64)
    T, H = x.shape
    b = x.reshape(T * H // 32, 32)
    codes = np.zeros(b.shape, dtype=np.uint8)
    scales = np.zeros(len(b), dtype=np.uint8)
    values = np.zeros(b.shape)
    limit, low, high, offset = ((448.0, -126, 120, 127) if format == "e4m3"
                                else (127.0, -126, 121, 133))
    for i, row in enumerate(b):
        if not np.isfinite(row).all():
            scales[i] = 255
            values[i] = np.nan
            continue
        S = low
        while S < high and np.abs(row).max() > np.ldexp(limit, S):
            S += 1
        y = np.ldexp(row, -S)
        if format == "e4m3":
            cap = 240.0 if S == 120 else 448.0
            q = round_e4m3(np.clip(y, -cap, cap))
            codes[i] = [_e4m3_code(v, np.signbit(r)) for v, r in zip(q, row)]
        else:
            q = np.clip(np.rint(y), -127, 127)
            codes[i] = q.astype(np.int8).view(np.uint8)
        scales[i] = S + offset
        values[i] = np.ldexp(q, S)
    return codes.reshape(T, H), scales.reshape(T, H // 32), values.reshape(T, H)


def _e4m3_code(v, negative):
    """The E4M3 bit pattern of a representable value."""
    a = abs(v)
    if a < 2.0 ** -6:
        code = int(a * 512)
    else:
        _, e = np.frexp(a)
        code = ((e - 1 + 7) << 3) | (int(a * 2.0 ** (4 - e)) - 8)
    return code | (0x80 if negative else 0)
