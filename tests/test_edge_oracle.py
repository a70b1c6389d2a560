"""The fp64 oracle of the operators at the block's edge, pinned by central differences of its own
forward and by the formats' definitions."""

import numpy as np
import pytest

from oracle import edge_oracle as O

ROUTINGS = [
    dict(k=3, scores="softmax", renormalize=True, scale=1.0),
    dict(k=3, scores="softmax", renormalize=False, scale=2.5),
    dict(k=3, scores="sigmoid", renormalize=True, scale=2.5),
    dict(k=3, scores="sigmoid", renormalize=False, scale=1.0),
    dict(k=3, scores="sigmoid", renormalize=True, scale=0.5, groups=4, top_groups=2, group_best=2),
]


@pytest.mark.parametrize("cfg", ROUTINGS)
def test_route_gradient_matches_differences(cfg):
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((4, 12))
    bias = rng.standard_normal(12) * 0.05
    dw = rng.standard_normal((4, 3))
    idx, w = O.route(logits, bias=bias, **cfg)
    kw = {n: cfg[n] for n in ("scores", "renormalize", "scale")}
    d = O.route_backward(logits, idx, w, dw, **kw)
    eps = 1e-6
    for t in range(4):
        for e in range(12):
            out = []
            for sign in (1, -1):
                l = logits.copy()
                l[t, e] += sign * eps
                i2, w2 = O.route(l, bias=bias, **cfg)
                assert np.array_equal(i2, idx)  # no decision within reach of the step
                out.append((w2 * dw).sum())
            assert (out[0] - out[1]) / (2 * eps) == pytest.approx(d[t, e], rel=1e-6, abs=1e-8)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_matches_differences(kind):
    rng = np.random.default_rng(4)
    x, dn = rng.standard_normal((3, 10)), rng.standard_normal((3, 10))
    w, b = rng.standard_normal(10), rng.standard_normal(10)
    dx, dw, db = O.norm_backward(dn, x, w, kind)
    loss = lambda x, w, b: float((O.norm(x, w, b, kind)[0] * dn).sum())  # noqa: E731
    eps = 1e-6
    for i in range(10):
        e = np.zeros(10)
        e[i] = eps
        assert (loss(x, w + e, b) - loss(x, w - e, b)) / (2 * eps) == pytest.approx(dw[i], rel=1e-6, abs=1e-7)
        assert (loss(x, w, b + e) - loss(x, w, b - e)) / (2 * eps) == pytest.approx(db[i], rel=1e-6, abs=1e-7)
        for t in range(3):
            xp, xm = x.copy(), x.copy()
            xp[t, i] += eps
            xm[t, i] -= eps
            assert (loss(xp, w, b) - loss(xm, w, b)) / (2 * eps) == pytest.approx(dx[t, i], rel=1e-6, abs=1e-7)


def _e4m3_value(code):
    e, m = (code >> 3) & 15, code & 7
    a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -a if code & 0x80 else a


@pytest.mark.parametrize("format", ["e4m3", "int8"])
def test_checkpoint_codes_stand_for_the_nearest_values(format):
    """Codes and scale bytes read back by the formats' definitions give the values, every value
    is a nearest element of its block's grid, and the scale is the smallest that holds it."""
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((6, 64)) * 2.0 ** rng.integers(-20, 20, (6, 1))).astype(np.float32)
    x[1, :32] = 0.0
    x[2, 5] = -0.0
    codes, scales, values = O.checkpoint(x, format)
    for t in range(6):
        for h in range(64):
            c, byte = int(codes[t, h]), int(scales[t, h // 32])
            if format == "e4m3":
                v = _e4m3_value(c) * 2.0 ** (byte - 127)
                grid = [_e4m3_value(q) * 2.0 ** (byte - 127) for q in range(127)]
            else:
                v = (c - 256 if c > 127 else c) / 64 * 2.0 ** (byte - 127)
                grid = [q / 64 * 2.0 ** (byte - 127) for q in range(128)]
            assert v == values[t, h]
            assert abs(abs(float(x[t, h])) - abs(v)) <= min(abs(abs(float(x[t, h])) - q) for q in grid)
        for blk in range(2):
            most = np.abs(x[t, 32 * blk:32 * blk + 32]).max()
            if most > 0:
                limit = 448.0 if format == "e4m3" else 127.0
                S = int(scales[t, blk]) - (127 if format == "e4m3" else 133)
                assert limit * 2.0 ** (S - 1) < most <= limit * 2.0 ** S


def test_masked_rows_and_ties():
    inf = np.inf
    logits = np.array([[-inf, -inf, -inf, -inf], [1.0, 1.0, 1.0, 0.0], [np.nan, 2.0, -inf, O.LOWEST],
                       [inf, 0.0, inf, 1.0]])
    idx, w = O.route(logits, 2)
    assert idx.tolist() == [[0, 1], [0, 1], [1, 0], [0, 2]]
    np.testing.assert_allclose(w, [[0, 0], [.5, .5], [1, 0], [.5, .5]])
