"""Sizes beyond 32 bits at the wrappers of the operators at the block's edge: refused, not taken for
what is left of them in 32 bits (no GPU; tensors without memory)."""

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from mxfp4_quantized_moe_b200 import build
    build.build()
    from mxfp4_quantized_moe_b200 import moe as m
    return m


WIDE = 2 ** 32 + 5


def test_scratch_of_more_rows_than_32_bits_hold(moe):
    assert moe.norm_workspace_bytes(2 ** 31 - 1, 64) > 0
    for T in (2 ** 31, WIDE):
        with pytest.raises(ValueError, match="32 bits"):
            moe.norm_workspace_bytes(T, 64)


@pytest.mark.parametrize("bad", [dict(k=WIDE), dict(groups=2 ** 32 + 1), dict(top_groups=2 ** 32 + 1),
                                 dict(group_best=2 ** 32 + 1)])
def test_routing_numbers(moe, bad):
    r = moe.Routing(**{"k": 2, **bad})
    with pytest.raises(ValueError, match="32 bits"):
        r.dims(4, 8)
    with pytest.raises(ValueError, match="32 bits"):
        moe.Routing(2).dims(WIDE, 8)


def test_rows(moe):
    x = torch.empty(WIDE, 32, dtype=torch.bfloat16, device="meta")
    cp = moe.Checkpoint(torch.empty(WIDE, 32, dtype=torch.uint8, device="meta"),
                        torch.empty(WIDE, 1, dtype=torch.uint8, device="meta"))
    v = torch.empty(WIDE, device="meta")
    calls = (lambda: moe.norm_forward(x), lambda: moe.norm_forward(cp),
             lambda: moe.norm_backward(x, x, v, v), lambda: moe.norm_backward(x, cp, v, v),
             lambda: moe.checkpoint_pack(x), lambda: moe.checkpoint_unpack(cp),
             lambda: moe.route(moe.Routing(2), torch.empty(WIDE, 8, device="meta")),
             lambda: moe.route_backward(moe.Routing(2), torch.empty(WIDE, 8, device="meta"), v, v, v))
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()
