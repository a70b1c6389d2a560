"""Expert routing on the GPU against the fp64 oracle (oracle/edge_oracle.py).

Indices are compared exactly: ties go to the lower index, and orders that fp32 keys cannot decide
are decided on fp64 keys.  Weights carry fp32 rounding only.  With r = 2^-24 (half a step of
fp32): log s_j is off by at most 3 r |log s_j|, the exponent's subtraction by r |.|, expf by 4 r,
the sum of the k terms by 8 r (a tree of shuffles), division and scaling by 2 r, so a weight is
within (24 + 16 max|l|) r of its value, relative.
"""

import numpy as np
import pytest
import torch

from oracle import edge_oracle as O

pytestmark = pytest.mark.gpu
R = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mxfp4_quantized_moe_b200 import moe as m
    return m


def oracle_args(r):
    return dict(scores=r.scores, groups=r.groups, top_groups=r.top_groups,
                group_best=r.group_best, renormalize=r.renormalize, scale=r.scale)


def weight_bound(logits):
    fin = logits[np.isfinite(logits) & (np.abs(logits) < 1e30)]
    return (24 + 16 * (np.abs(fin).max() if fin.size else 0.0)) * R


def check(moe, r, logits, bias, seed=0):
    logits = logits.float()
    l64 = logits.double().numpy()
    T, E = logits.shape
    counts = torch.full((E,), -7, dtype=torch.int32, device="cuda")
    lc, bc = logits.cuda(), None if bias is None else bias.float().cuda()
    idx, w = moe.route(r, lc, bc, counts=counts)
    ri, rw = O.route(l64, r.k, None if bias is None else bias.double().numpy(), **oracle_args(r))
    assert idx.dtype == torch.int32 and np.array_equal(idx.cpu().numpy(), ri)
    gw = w.double().cpu().numpy()
    rel = weight_bound(l64)
    assert np.all(np.abs(gw - rw) <= rel * np.abs(rw) + 1e-37), np.abs(gw - rw).max()
    assert np.array_equal(gw == 0, rw == 0) or rw.min() < 1e-37
    assert np.array_equal(counts.cpu().numpy(), np.bincount(ri.ravel(), minlength=E))

    dw = torch.randn(T, r.k, generator=torch.Generator().manual_seed(seed))
    d = moe.route_backward(r, lc, idx, w, dw.cuda()).double().cpu().numpy()
    d64 = dw.double().numpy()
    ref = O.route_backward(l64, ri, gw, d64, r.scores, r.renormalize, r.scale)
    # every term of an entry, in magnitude: each carries the weights' and the scores' rounding
    part = np.abs(gw * d64)
    mag = np.zeros((T, E))
    for t in range(T):
        np.add.at(mag[t], ri[t], part[t] + np.abs(gw[t]) * part[t].sum() / abs(r.scale))
    if r.scores == "softmax" and not r.renormalize:
        mag += np.stack([O._scores(row, "softmax")[0] for row in l64]) * part.sum(1, keepdims=True)
    assert np.all(np.abs(d - ref) <= 4 * rel * mag + 1e-37), np.abs(d - ref).max()
    return idx, w


def normal(T, E, seed, scale=1.5):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * scale


SHAPES = [(1, 1, 1), (1, 32, 4), (3, 2, 2), (7, 5, 3), (33, 32, 4), (9, 33, 8), (20, 64, 64),
          (65, 100, 7), (40, 128, 4), (5, 200, 33), (70, 256, 8), (2, 256, 256)]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route(moe, T, E, k, scores, renormalize, biased):
    bias = normal(1, E, 11, 0.05)[0] if biased else None
    r = moe.Routing(k, scores, renormalize=renormalize, scale=1.0 if renormalize else 2.5)
    check(moe, r, normal(T, E, T + E), bias)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,best,k", [
    (256, 8, 4, 2, 8), (256, 8, 8, 2, 8), (256, 32, 3, 1, 8), (160, 8, 3, 1, 6), (64, 2, 1, 2, 32),
    (30, 5, 2, 2, 12), (12, 12, 4, 1, 4), (60, 4, 2, 2, 5), (2, 2, 1, 1, 1)])
def test_route_groups(moe, E, groups, top_groups, best, k, scores, biased):
    bias = normal(1, E, 12, 0.05)[0] if biased else None
    r = moe.Routing(k, scores, groups, top_groups, best, scale=2.5)
    check(moe, r, normal(57, E, E + groups), bias)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_equal_logits_go_to_the_lower_index(moe, scores, groups):
    """Logits on a coarse grid: most rows hold exact ties, inside the selection and at its end."""
    logits = torch.round(normal(200, 64, 5) * 2) / 2
    r = moe.Routing(6, scores, groups, min(groups, 2), 2 if groups > 1 else 1)
    check(moe, r, logits, None)
    check(moe, r, logits, torch.zeros(64))
    check(moe, r, logits, torch.round(normal(1, 64, 6)[0] * 2) / 16)
    check(moe, r, torch.zeros(3, 64), None)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
def test_keys_closer_than_fp32_can_tell(moe, scores, groups):
    """Pairs of experts whose keys differ by less than an fp32 step of the key, in both orders:
    the score falls by what the bias rises, up to the bias's own rounding."""
    T, E = 64, 64
    logits = normal(T, E, 8, 0.5)
    bias = torch.zeros(E)
    if scores == "sigmoid":
        s = lambda v: 1.0 / (1.0 + torch.exp(-v))  # noqa: E731
        for e in range(0, E, 2):
            logits[:, e] = 1.0 + 0.01 * e
            logits[:, e + 1] = logits[:, e] - 0.25
            l = logits[0].double()
            bias[e + 1] = (s(l[e]) - s(l[e + 1])).float()
    else:
        logits = logits[:1].repeat(T, 1)
        p = torch.softmax(logits[0].double(), 0)
        bias = (p.max() - p).float()  # every key is the largest score, up to rounding
    r = moe.Routing(8, scores, groups, max(1, groups // 2), 2 if groups > 1 else 1)
    check(moe, r, logits, bias)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_experts(moe, scores, renormalize, groups, biased):
    """-inf, the lowest finite value and NaN mask an expert; rows left with fewer than k experts,
    with one and with none fill up with weights of exactly 0."""
    E, k = 40, 6
    logits = normal(12, E, 9)
    low = torch.finfo(torch.float32).min
    for t, v in enumerate([float("-inf"), low, float("nan")] * 4):
        keep = [E, 7, 5, 1, 0, 0][t // 2]
        at = torch.randperm(E, generator=torch.Generator().manual_seed(t))
        logits[t, at[keep:]] = v
    bias = None
    if biased:
        bias = normal(1, E, 10, 0.05)[0]
        bias[3], bias[17], bias[30] = float("-inf"), low, float("nan")
    r = moe.Routing(k, scores, groups, min(groups, 2), 2 if groups > 1 else 1, renormalize, 2.5)
    idx, w = check(moe, r, logits, bias)
    assert torch.isfinite(w).all() and (w[8:] == 0).all()


def test_extreme_logits(moe):
    """Scores that underflow still share the weight by their ratio; +inf is the largest value."""
    logits = torch.tensor([[-200.0, -201.0, -300.0, -500.0], [float("inf"), 0.0, float("inf"), 1.0],
                           [3e38, -3e38, 0.0, 1.0], [90.0, 89.0, -90.0, 0.0]])
    for scores in ("softmax", "sigmoid"):
        r = moe.Routing(2, scores)
        idx, w = moe.route(r, logits.cuda())
        ri, rw = O.route(logits.double().numpy(), 2, scores=scores)
        assert np.array_equal(idx.cpu().numpy(), ri)
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=16 * 300 * R)
        d = moe.route_backward(r, logits.cuda(), idx, w, torch.ones(4, 2, device="cuda"))
        assert torch.isfinite(d).all()


def test_backward_takes_any_slots(moe):
    """A caller's own slots: an expert twice in a row receives the sum, an index outside [0, E)
    nothing."""
    logits = normal(3, 8, 1)
    idx = torch.tensor([[1, 1, 3], [0, 9, 2], [-1, 5, 5]], dtype=torch.int32)
    w = torch.tensor([[.5, .25, .25], [.5, .25, .25], [.2, .4, .4]])
    dw = normal(3, 3, 2)
    for scores in ("softmax", "sigmoid"):
        for renorm in (True, False):
            r = moe.Routing(3, scores, renormalize=renorm)
            d = moe.route_backward(r, logits.cuda(), idx.cuda(), w.cuda(), dw.cuda())
            p, dot = w.double(), (w.double() * dw.double()).sum(1, keepdim=True)
            q = p * (dw.double() - dot) if renorm else p * dw.double()
            ref = torch.zeros(3, 8, dtype=torch.float64)
            for t in range(3):
                for j in range(3):
                    e = int(idx[t, j])
                    if 0 <= e < 8:
                        f = 1 / (1 + logits[t, e].double().exp()) if scores == "sigmoid" else 1.0
                        ref[t, e] += q[t, j] * f
            if scores == "softmax" and not renorm:
                ref -= torch.softmax(logits.double(), 1) * dot
            np.testing.assert_allclose(d.double().cpu().numpy(), ref.numpy(), rtol=2e-6, atol=2e-6)


@pytest.mark.parametrize("k", [7, 12, 40])
def test_backward_adds_repeated_slots_in_order(moe, k):
    """Rows that name few experts many times: the same bits every time, the sum of the slots."""
    T, E = 33, 48
    gen = torch.Generator().manual_seed(k)
    logits, dw = normal(T, E, 1), normal(T, k, 2)
    idx = torch.randint(0, 3, (T, k), generator=gen, dtype=torch.int32) * 7
    w = torch.rand(T, k, generator=gen)
    r = moe.Routing(k, "softmax")
    args = (r, logits.cuda(), idx.cuda(), w.cuda(), dw.cuda())
    d = moe.route_backward(*args)
    assert all(torch.equal(d, moe.route_backward(*args)) for _ in range(3))
    q = w.double() * (dw.double() - (w.double() * dw.double()).sum(1, keepdim=True))
    ref = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, idx.long(), q)
    mag = torch.zeros(T, E, dtype=torch.float64).scatter_add_(
        1, idx.long(), w.double() * (dw.double().abs() + (w * dw).double().abs().sum(1, keepdim=True)))
    # products, the dot over k terms and the sum of at most k slots, each rounded once
    assert ((d.double().cpu() - ref).abs() <= (2 * k + 8) * R * mag + 1e-30).all()


def test_rows_past_32_bit_offsets(moe):
    """Logits of more than 2^31 elements: the last tokens as in a batch of their own."""
    E, k = 256, 4
    T = 2 ** 31 // E + 1000
    logits = torch.empty(T, E, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    r = moe.Routing(k, "softmax", renormalize=False)
    idx, w = moe.route(r, logits)
    tail = logits[-999:].clone()
    i2, w2 = moe.route(r, tail)
    assert torch.equal(idx[-999:], i2) and torch.equal(w[-999:], w2)
    dw = torch.ones(T, k, device="cuda")
    d = moe.route_backward(r, logits, idx, w, dw)
    assert torch.equal(d[-999:], moe.route_backward(r, tail, i2, w2, dw[:999].contiguous()))


def test_empty_and_large_batches(moe):
    r = moe.Routing(2, "sigmoid")
    counts = torch.ones(8, dtype=torch.int32, device="cuda")
    idx, w = moe.route(r, torch.empty(0, 8, device="cuda"), counts=counts)
    assert idx.shape == w.shape == (0, 2) and not counts.any()
    assert moe.route_backward(r, torch.empty(0, 8, device="cuda"), idx, w, w).shape == (0, 8)
    logits = normal(20001, 16, 3)
    check(moe, r, logits, None)


def test_outputs_end_at_the_last_token(moe):
    """Rows behind the last token of larger buffers stay as they were."""
    T, E, k = 37, 48, 5
    logits = normal(T, E, 4).cuda()
    for r in (moe.Routing(k, "sigmoid"), moe.Routing(k, "softmax", renormalize=False)):
        idx = torch.full((T + 3, k), -5, dtype=torch.int32, device="cuda")
        w = torch.full((T + 3, k), 7.0, device="cuda")
        d = torch.full((T + 3, E), 7.0, device="cuda")
        moe.route(r, logits, topk_idx=idx[:T], topk_w=w[:T])
        moe.route_backward(r, logits, idx[:T], w[:T], torch.ones(T, k, device="cuda"), d[:T])
        assert (idx[T:] == -5).all() and (w[T:] == 7).all() and (d[T:] == 7).all()
        assert (idx[:T] >= 0).all()


def test_rows_without_vector_alignment(moe):
    """Views that begin at any fp32 element, and E that no vector width divides."""
    for E in (64, 61):
        base = normal(1, 40 * E + 3, 5)[0].cuda()
        for off in (1, 2, 3):
            logits = base[off:off + 40 * E].view(40, E)
            r = moe.Routing(4)
            idx, w = moe.route(r, logits)
            i2, w2 = moe.route(r, logits.clone())
            assert torch.equal(idx, i2) and torch.equal(w, w2)
            dw = torch.randn(40, 4, device="cuda")
            d = torch.zeros(40 * E + 3, device="cuda")[off:off + 40 * E].view(40, E)
            moe.route_backward(r, logits, idx, w, dw, d_logits=d)
            assert torch.equal(d, moe.route_backward(r, logits.clone(), i2, w2, dw))


def test_other_stream_and_captured_replay(moe):
    r = moe.Routing(4, "sigmoid", 4, 2, 2)
    logits, bias = normal(130, 64, 6).cuda(), normal(1, 64, 7, 0.05)[0].cuda()
    dw = torch.randn(130, 4, device="cuda")
    idx, w = moe.route(r, logits, bias)
    d = moe.route_backward(r, logits, idx, w, dw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    i2, w2 = moe.route(r, logits, bias, stream=s)
    d2 = moe.route_backward(r, logits, i2, w2, dw, stream=s)
    s.synchronize()
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(d, d2)
    counts = torch.zeros(64, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    static = logits.clone()
    with torch.cuda.graph(g):
        i3, w3 = moe.route(r, static, bias, counts=counts)
        d3 = moe.route_backward(r, static, i3, w3, dw)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, i3) and torch.equal(w, w3) and torch.equal(d, d3)
    assert int(counts.sum()) == 130 * 4
    static.copy_(normal(130, 64, 60))
    g.replay()
    i4, w4 = moe.route(r, static, bias)
    assert torch.equal(i3, i4) and torch.equal(w3, w4)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,k", [(4, 1, 2), (32, 4, 4), (40, 1, 8), (128, 8, 6), (64, 1, 12)])
def test_infinite_logits_without_renormalisation(moe, scores, E, groups, k):
    """+inf is the largest finite value: the softmax of a row that holds some is shared by them."""
    logits = normal(9, E, E)
    inf = float("inf")
    logits[0, 0] = logits[1, 1] = logits[1, E - 1] = logits[3, 2] = inf
    logits[2] = inf
    logits[4, 0], logits[4, 1:] = inf, -inf
    logits[5, 0], logits[5, 1] = 3e38, inf
    for best in (1, 2):
        r = moe.Routing(k, scores, groups, max(1, groups // 2), best if groups > 1 else 1, False, 2.5)
        for bias in (None, torch.zeros(E)):
            idx, w = moe.route(r, logits.cuda(), None if bias is None else bias.cuda())
            ri, rw = O.route(logits.double().numpy(), k, None if bias is None else bias.numpy(),
                             **oracle_args(r))
            assert np.array_equal(idx.cpu().numpy(), ri)
            # scores of ordinary rows as in check(); those of the infinite ones are 1, 1/n or 0
            np.testing.assert_allclose(w.double().cpu().numpy(), rw, rtol=weight_bound(logits.double().numpy()),
                                       atol=1e-37)
            d = moe.route_backward(r, logits.cuda(), idx, w, torch.ones(9, k, device="cuda"))
            assert torch.isfinite(d).all()


def test_exact_tie_beside_a_near_one(moe):
    """The last place is held by one of two equal experts, and the place before it by one whose key
    is off by less than fp32 tells: where the equal ones rank first, both are chosen."""
    T, E = 256, 32
    gen = torch.Generator().manual_seed(21)
    la = torch.rand(T, generator=gen) * 2 - 1
    key = torch.sigmoid(la.double()) + torch.tensor(0.05).double()
    lx = torch.log(key / (1 - key)).float()  # its key is the others' up to the rounding of lx
    logits = torch.full((T, E), -10.0) + normal(T, E, 22, 0.5)
    bias = torch.zeros(E)
    for x, a, b, k in ((1, 5, 6, 2), (9, 2, 30, 2), (31, 8, 24, 2)):
        rows, shift = logits.clone(), bias.clone()
        rows[:, x], rows[:, a], rows[:, b] = lx, la, la
        shift[a] = shift[b] = 0.05
        kx = torch.sigmoid(lx.double())
        first = kx < key
        assert 32 < int(first.sum()) < T - 32  # both orders
        for groups in (1, 4):
            check(moe, moe.Routing(k, "sigmoid", groups, groups), rows, shift)
            check(moe, moe.Routing(k, "sigmoid", groups, groups, renormalize=False), rows, shift)


def test_zero_weight_with_an_infinite_gradient(moe):
    """A slot of weight 0 has no gradient, whatever the other slots hold."""
    logits = normal(2, 16, 3)
    logits[:, 2:] = float("-inf")
    for k in (4, 12):
        for scores in ("softmax", "sigmoid"):
            r = moe.Routing(k, scores)
            idx, w = moe.route(r, logits.cuda())
            assert (w[:, 2:] == 0).all()
            dw = torch.ones(2, k, device="cuda")
            dw[1, 0] = float("inf")
            d = moe.route_backward(r, logits.cuda(), idx, w, dw)
            assert torch.isfinite(d[0]).all() and (d[:, 2:] == 0).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,best", [(1, 1), (4, 1), (4, 2)])
def test_saturated_scores_order_like_their_logits(moe, scores, groups, best):
    """Logits of which fp64 scores no longer tell the order (sigmoid(40) = sigmoid(50) = 1)."""
    for E, k in ((32, 4), (64, 8), (64, 12)):
        logits = torch.cat([normal(24, E, E, 4.0) + 60, normal(24, E, E + 1, 60.0)])
        check(moe, moe.Routing(k, scores, groups, max(1, groups // 2), best), logits, None)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(9, 8), (9, 4), (40, 8), (200, 6), (61, 12)])
def test_biases_far_above_the_scores(moe, scores, E, k):
    """Keys whose fp32 step is as wide as the scores: the order is that of the fp64 keys, and a
    masked expert beside the last one chosen stays out."""
    logits = normal(40, E, E)
    for t in range(0, 40, 2):
        logits[t, (3 * t) % E] = float("nan") if t % 4 else float("-inf")
    for level, spread in ((1e5, 5.0), (1e5, 0.0), (3e7, 0.0), (-2e4, 20.0)):
        bias = level + normal(1, E, 31)[0] * spread
        check(moe, moe.Routing(k, scores, renormalize=False), logits, bias)
