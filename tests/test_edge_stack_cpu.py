"""The stack with a norm, a routing and checkpoints, on the CPU (no GPU): its chaining run in fp64
on functions by definition, against central differences of its own forward, for the stack's
input and for the norms' parameters."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

from mxfp4_quantized_moe_b200.stack import MoeStack, StackBlock
from oracle import edge_oracle as O

T, H, E, K, L = 3, 32, 6, 2, 3


class FakeBlocks:
    """Experts as fixed linear maps with a tanh, differentiated by hand."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.W = rng.standard_normal((L, E, H, H)) * 0.2
        self.state = None

    def forward(self, l, x, how):
        idx, w = how
        y = np.tanh(np.einsum("th,tkgh->tkg", x.numpy(), self.W[l][idx.numpy()]))
        self.state = (l, x.numpy(), idx.numpy(), w.numpy(), y)
        return torch.from_numpy(np.einsum("tk,tkg->tg", w.numpy(), y))

    def backward(self, l, g):
        at, x, idx, w, y = self.state
        assert at == l  # the state is the block's own recomputed forward
        d_w = np.einsum("tg,tkg->tk", g.numpy(), y)
        d = w[:, :, None] * g.numpy()[:, None] * (1 - y * y)
        return torch.from_numpy(np.einsum("tkg,tkgh->th", d, self.W[l][idx])), None, torch.from_numpy(d_w)


def ops(calls):
    def norm_forward(x, w, b, *, kind, eps, y=None, checkpoint=None, dtype=None):
        rows = x["kept"] if isinstance(x, dict) else x
        x_out = None if y is None else rows + y
        rows = rows if y is None else x_out
        calls.append("norm")
        out, mean, rstd = O.norm(rows.numpy(), w.numpy(), None if b is None else b.numpy(), kind, eps)
        return SimpleNamespace(out=torch.from_numpy(out), x_out=x_out, mean=mean, rstd=rstd,
                               checkpoint={"kept": rows} if checkpoint else None)

    def norm_backward(d, x, mean, rstd, w, *, kind, g):
        rows = x["kept"] if isinstance(x, dict) else x
        dx, dw, db = O.norm_backward(d.numpy(), rows.numpy(), w.numpy(), kind, 1e-5, g.numpy())
        return torch.from_numpy(dx), torch.from_numpy(dw), torch.from_numpy(db)

    def route(r, logits, bias):
        idx, w = O.route(logits.numpy(), K, None if bias is None else bias.numpy(), scores=r.scores,
                         renormalize=r.renormalize, scale=r.scale)
        return torch.from_numpy(idx), torch.from_numpy(w)

    def route_backward(r, logits, idx, w, d_w):
        return torch.from_numpy(O.route_backward(logits.numpy(), idx.numpy(), w.numpy(), d_w.numpy(),
                                                 r.scores, r.renormalize, r.scale))

    return SimpleNamespace(norm_forward=norm_forward, norm_backward=norm_backward, route=route,
                           route_backward=route_backward,
                           checkpoint_pack=lambda x, f: calls.append("pack") or {"kept": x},
                           checkpoint_unpack=lambda c, dtype: calls.append("unpack") or c["kept"])


def residual_router(x, y, w_r, b_r):
    x_next = None if y is None else x + y
    return x_next, None if w_r is None else (x if y is None else x_next) @ w_r + b_r


def grad_chain(g, dx, d_logits, w_r):
    return g + (0.0 if dx is None else dx) + d_logits @ w_r.T


def stack(norm, scores, checkpoint, seed=5):
    rng = np.random.default_rng(seed)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s))  # noqa: E731
    blocks = [StackBlock(None, None, draw(H, E) * 0.3, draw(E) * 0.1,
                         1 + 0.2 * draw(H) if norm else None, 0.2 * draw(H) if norm == "layer" else None,
                         0.05 * draw(E)) for _ in range(L)]
    fake, calls = FakeBlocks(seed), []
    routing = SimpleNamespace(k=K, scores=scores, renormalize=True, scale=1.5)
    st = MoeStack(None, blocks, block_forward=fake.forward, block_backward=fake.backward,
                  residual_router=residual_router, grad_chain=grad_chain, norm=norm,
                  routing=routing, checkpoint=checkpoint, ops=ops(calls))
    return st, draw(T, H), draw(T, H), calls


@pytest.mark.parametrize("norm", [None, "layer", "rms"])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("checkpoint", [None, "e4m3"])
def test_gradient_of_the_stack_matches_differences(norm, scores, checkpoint):
    st, x, dy, calls = stack(norm, scores, checkpoint)

    def loss(x0):
        out, saved = st.forward(x0)
        return float((out * dy).sum()), saved

    _, saved = loss(x)
    assert len(saved) == L and all(len(s) == 4 for s in saved)
    assert all(isinstance(s[0], dict) == bool(checkpoint) for s in saved)
    if checkpoint and not norm:
        assert calls.count("pack") == L
    g = st.backward(dy, saved)
    eps, rng = 1e-6, np.random.default_rng(1)
    picks = [s[2].numpy() for s in saved]

    def check(got, move):
        up, s1 = move(eps)
        down, s2 = move(-eps)
        assert all(np.array_equal(a, s[2]) and np.array_equal(a, b[2])
                   for a, s, b in zip(picks, s1, s2))  # no expert within reach of the step
        assert (up - down) / (2 * eps) == pytest.approx(got, rel=1e-5, abs=1e-7)

    for _ in range(10):
        t, h = rng.integers(T), rng.integers(H)

        def at(e):
            x1 = x.clone()
            x1[t, h] += e
            return loss(x1)
        check(float(g[t, h]), at)
    if norm:
        assert len(st.norm_grads) == L
        grads = st.norm_grads
        for l in range(L):
            for p, d in ((st.blocks[l].norm_w, grads[l][0]), (st.blocks[l].norm_b, grads[l][1])):
                if p is None:
                    continue
                h = int(rng.integers(H))

                def at(e):
                    p[h] += e
                    out = loss(x)
                    p[h] -= e
                    return out
                check(float(d[h]), at)


def test_a_routing_of_another_k_is_refused():
    with pytest.raises(ValueError):
        MoeStack(SimpleNamespace(k=4), [], block_forward=lambda *a: None, block_backward=lambda *a: None,
                 residual_router=residual_router, grad_chain=grad_chain,
                 routing=SimpleNamespace(k=2), ops=SimpleNamespace())
