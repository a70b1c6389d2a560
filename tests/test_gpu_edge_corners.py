"""Corners of the operators at the block's edge on the GPU: calls that the documentation allows
and that ordinary batches do not reach, against the fp64 oracle or the entry points themselves.
"""

import numpy as np
import pytest
import torch

from test_gpu_norm import R, TYPES, f64, rows
from test_gpu_routing import check, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mxfp4_quantized_moe_b200 import moe as m
    return m


# ---- routing: groups whose largest keys cancel ----------------------------------------------
def cancelling(E, groups, level, plain=0):
    """A balance bias of +level on one expert of each group and -level on another; the last
    `plain` groups have none."""
    size = E // groups
    bias = normal(1, E, 41, 0.05)[0].view(groups, size)
    bias[:groups - plain, 0] += level
    bias[:groups - plain, 1] -= level
    return bias.reshape(E)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("level", [100.0, 1e4, 1e5])
@pytest.mark.parametrize("E,groups,top_groups,k", [(32, 16, 8, 4), (4, 2, 1, 2), (160, 8, 3, 6)])
def test_group_sums_of_keys_that_cancel(moe, E, groups, top_groups, k, level, scores):
    """The sum of two keys of opposite sign is small, its rounding error is not: groups are ranked
    on fp64 keys wherever that error could change their order."""
    logits = normal(1500, E, E)
    size = E // groups
    if size > 2:  # only the two remain, so that they are the group's largest keys
        logits.view(-1, groups, size)[:, :, 2:] = float("-inf")
    r = moe.Routing(k, scores, groups, top_groups, 2, renormalize=False)
    check(moe, r, logits, cancelling(E, groups, level))
    check(moe, r, logits, cancelling(E, groups, level, plain=groups // 2))


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("level", [100.0, 1e4, 1e5])
@pytest.mark.parametrize("E,groups,top_groups,k", [(32, 4, 1, 1), (64, 8, 4, 2), (64, 4, 2, 2),
                                                   (40, 5, 2, 1), (256, 8, 4, 4)])
def test_group_sums_of_keys_that_cancel_in_whole_slots(moe, E, groups, top_groups, k, level, scores):
    """The same for groups of whole slots, few of whose experts are chosen (the keys of those are
    far apart, and do not send the row to fp64 themselves)."""
    logits = normal(1500, E, E + 1)
    logits.view(-1, groups, E // groups)[:, :, 2:] = float("-inf")
    r = moe.Routing(k, scores, groups, top_groups, 2, renormalize=False)
    check(moe, r, logits, cancelling(E, groups, level))
    check(moe, r, logits, cancelling(E, groups, level, plain=groups // 2))


@pytest.mark.parametrize("E,groups,k", [(32, 4, 1), (16, 8, 2)])
def test_group_sums_beside_the_largest_values(moe, E, groups, k):
    """Biases up to the largest finite value: sums that fp32 no longer holds are in order, and a
    group without experts stays behind all others."""
    top = torch.finfo(torch.float32).max
    logits = normal(64, E, E)
    size = E // groups
    logits.view(-1, groups, size)[::2, 1] = float("-inf")
    bias = torch.zeros(groups, size)
    bias[0, :2] = torch.tensor([top, top / 2])
    bias[1, :2] = torch.tensor([top, top])
    bias[2, :2] = torch.tensor([top, -top / 2])
    bias[3] = -top / 2
    for n in (1, 2, 3):
        r = moe.Routing(k, "sigmoid", groups, n, 2, renormalize=False)
        check(moe, r, logits, bias.reshape(E))


# ---- the norm's gradients of rows far from zero ---------------------------------------------
@pytest.mark.parametrize("H", [64, 512, 4384])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value,eps", [(2.0 ** 114, 1e-12), (2.0 ** 114, 1e-5), (-2.0 ** 100, 1e-20)])
def test_gradient_of_constant_rows_of_large_values(moe, H, dtype, value, eps):
    """A constant row has x_hat = 0 whatever its mean: dx = rstd (v - mean v).  Lanes past the
    row's end hold no features, and mean * rstd, which may be beyond fp32, is no part of it."""
    dt = TYPES[dtype]
    mean = torch.full((3,), value, device="cuda")
    rstd = torch.full((3,), eps ** -0.5, device="cuda")
    d, g = rows(3, H, dt, 1).cuda(), rows(3, H, dt, 2).cuda()
    v, r = f64(d), f64(rstd)[:, None]
    for off in (0, 1, None):  # in place, without vector alignment, from a checkpoint
        x = torch.full((3 * H + 8,), value, dtype=dt, device="cuda")[off or 0:][:3 * H].view(3, H)
        if off is None:
            x = moe.checkpoint_pack(x)
        if H & (H - 1) == 0:  # the mean is exact
            f = moe.norm_forward(x, eps=eps, dtype=dt)
            assert not f.out.any() and torch.equal(f.mean, mean)
        for grad in (None, g):
            dx, dw, db = moe.norm_backward(d, x, mean, rstd, g=grad)
            ref = (v - v.mean(1, keepdims=True)) * r
            mag = (np.abs(v) + np.abs(v).mean(1, keepdims=True)) * r
            if grad is not None:
                ref, mag = ref + f64(grad), mag + np.abs(f64(grad))
            # the mean's sum and product, the two products and the sum with g
            tol = 80 * R * mag
            tol = tol + torch.finfo(dt).eps / 2 * (np.abs(ref) + tol)
            assert np.all(np.abs(f64(dx) - ref) <= tol)
            assert not dw.any()
            assert np.all(np.abs(f64(db) - v.sum(0)) <= 4 * R * np.abs(v).sum(0))
