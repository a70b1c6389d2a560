"""Host-side checks of the operators at the block's edge (no GPU): the C ABI refuses bad arguments
before it touches a device, its structs match the binding's, and the wrappers refuse tensors of
the wrong shape, type, layout or place."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, F, G = (ctypes.c_void_p((1 << 20) + (i << 18)) for i in range(6))  # never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    from mxfp4_quantized_moe_b200 import build
    build.build()
    from mxfp4_quantized_moe_b200 import _lib
    return _lib


@pytest.fixture(scope="module")
def reached(L):
    """What a valid call returns here: without a GPU it gets as far as the device check."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible: the made-up pointers below would reach a launch")
    return (L.ERR_CUDA, L.ERR_UNSUPPORTED_DEVICE)


def test_structs_match_the_header(L):
    src = open(os.path.join(ROOT, "include", "mxfp4_moe.h")).read()
    for name, cls in (("routing", L.Routing), ("checkpoint", L.Checkpoint), ("norm", L.Norm)):
        body = re.search(r"typedef struct \{([^}]*)\} mxfp4_moe_%s;" % name, src).group(1)
        assert re.findall(r"(\w+)\s*[,;]", body) == [f[0] for f in cls._fields_]
    consts = dict(re.findall(r"#define MXFP4_MOE_((?:SCORES|CHECKPOINT|NORM|ROWS)_\w+) (\d+)", src))
    for prefix, table in (("SCORES", L.SCORES), ("CHECKPOINT", L.CHECKPOINTS), ("NORM", L.NORMS)):
        assert {n.split("_")[1].lower(): int(v) for n, v in consts.items()
                if n.startswith(prefix + "_")} == table
    assert (int(consts["ROWS_BF16"]), int(consts["ROWS_FP32"])) == (L.ROWS_BF16, L.ROWS_FP32)


GOOD = dict(T=4, E=16, k=4, scores=0, groups=4, top_groups=2, group_best=2, renormalize=1, scale=1.0)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=257, groups=1, top_groups=1), dict(k=0), dict(k=17), dict(scores=2),
    dict(scores=-1), dict(groups=0), dict(groups=3), dict(groups=64), dict(top_groups=0),
    dict(top_groups=5), dict(top_groups=1, k=5), dict(group_best=0), dict(group_best=3),
    dict(groups=16, top_groups=4, group_best=2), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=1e-40)])
def test_routing_refusals(L, bad):
    r = L.Routing(*(dict(GOOD, **bad)[n] for n, _ in L.Routing._fields_))
    assert L.lib.mxfp4_moe_route(r, A, None, B, C, None, None) == L.ERR_INVALID_ARG
    assert L.lib.mxfp4_moe_route_backward(r, A, B, C, D, F, None) == L.ERR_INVALID_ARG


def test_routing_pointers(L, reached):
    r = L.Routing(*(GOOD[n] for n, _ in L.Routing._fields_))
    f, b = L.lib.mxfp4_moe_route, L.lib.mxfp4_moe_route_backward
    for args in [(None, None, B, C, None), (A, None, None, C, None), (A, None, B, None, None),
                 (ODD, None, B, C, None), (A, ODD, B, C, None), (A, None, ODD, C, None),
                 (A, None, B, ODD, None), (A, None, B, C, ODD), (A, None, A, C, None),
                 (A, None, B, B, None), (A, B, B, C, None), (A, None, B, C, C)]:
        assert f(r, *args, None) == L.ERR_INVALID_ARG, args
    assert f(None, A, None, B, C, None, None) == L.ERR_INVALID_ARG
    assert f(r, A, D, B, C, F, None) in reached
    for args in [(None, B, C, D, F), (A, None, C, D, F), (A, B, None, D, F), (A, B, C, None, F),
                 (A, B, C, D, None), (A, B, C, D, ODD), (A, B, C, D, A), (A, B, C, D, D)]:
        assert b(r, *args, None) == L.ERR_INVALID_ARG, args
    assert b(r, A, B, C, D, F, None) in reached


def test_forward_routed_refusals(L, reached):
    d, w = L.Dims(4, 64, 64, 4, 2, 1.702, 7.0, 0), L.Weights(A, A, A, A, A, A)
    n = ctypes.c_size_t()
    assert L.lib.mxfp4_moe_workspace_size(d, n) == 0
    f = L.lib.mxfp4_moe_forward_routed
    for args in [(None, B, C, D, F, n.value), (A, None, C, D, F, n.value), (A, B, None, D, F, n.value),
                 (A, B, C, None, F, n.value), (A, B, C, D, None, n.value), (A, ODD, C, D, F, n.value),
                 (ODD, B, C, D, F, n.value)]:
        assert f(d, w, *args, None) == L.ERR_INVALID_ARG, args
    assert f(d, w, A, B, C, D, F, n.value - 1, None) == L.ERR_WORKSPACE_TOO_SMALL
    assert f(d, L.Weights(), A, B, C, D, F, n.value, None) == L.ERR_INVALID_ARG
    assert f(d, w, A, B, C, D, F, n.value, None) in reached


def test_checkpoint_refusals(L, reached):
    cp = L.Checkpoint(B, C, 0)
    for f, swap in ((L.lib.mxfp4_moe_checkpoint_pack, False), (L.lib.mxfp4_moe_checkpoint_unpack, True)):
        def call(T, H, fmt, x, c):
            return f(T, H, fmt, c, x, None) if swap else f(T, H, fmt, x, c, None)
        for args in [(-1, 64, 0, A, cp), (4, 48, 0, A, cp), (4, 0, 0, A, cp), (4, 16416, 0, A, cp),
                     (4, 64, 2, A, cp), (4, 64, 0, None, cp), (4, 64, 0, ODD, cp), (4, 64, 0, A, None),
                     (4, 64, 0, A, L.Checkpoint(None, C, 0)), (4, 64, 0, A, L.Checkpoint(B, None, 0)),
                     (4, 64, 0, A, L.Checkpoint(ODD, C, 0)), (4, 64, 0, A, L.Checkpoint(B, C, 2)),
                     (4, 64, 0, A, L.Checkpoint(A, C, 0)), (4, 64, 0, A, L.Checkpoint(B, A, 0))]:
            assert call(*args) == L.ERR_INVALID_ARG, args
        assert call(4, 64, 1, A, cp) in reached
    assert L.lib.mxfp4_moe_checkpoint_pack(4, 64, 0, A, L.Checkpoint(B, B, 0), None) == L.ERR_INVALID_ARG


def test_norm_refusals(L, reached):
    ok = L.Norm(4, 64, 0, 1e-5, 0, 0)
    f, b, size = (L.lib.mxfp4_moe_norm_forward, L.lib.mxfp4_moe_norm_backward,
                  L.lib.mxfp4_moe_norm_workspace_size)
    n = ctypes.c_size_t()
    for bad in [(-1, 64, 0, 1e-5, 0, 0), (4, 0, 0, 1e-5, 0, 0), (4, 16385, 0, 1e-5, 0, 0),
                (4, 64, 2, 1e-5, 0, 0), (4, 64, 0, -1.0, 0, 0), (4, 64, 0, float("nan"), 0, 0),
                (4, 64, 0, 1e-5, 2, 0), (4, 64, 0, 1e-5, 0, -1)]:
        d = L.Norm(*bad)
        assert f(d, A, None, None, None, None, None, None, B, C, D, None) == L.ERR_INVALID_ARG
        assert b(d, A, B, None, C, D, None, None, F, None, None, None, 0, None) == L.ERR_INVALID_ARG
        assert size(d, n) == L.ERR_INVALID_ARG
    cp = L.Checkpoint(F, G, 0)
    #     x, from, y, weight, bias, x_out, to, out, mean, rstd
    for args in [(None, None, None, None, None, None, None, B, C, D),   # no rows
                 (A, cp, None, None, None, None, None, B, C, D),        # rows twice
                 (A, None, B, None, None, None, None, C, None, D),      # y without x_out
                 (A, None, None, None, None, B, None, C, None, D),      # x_out without y
                 (None, cp, A, None, None, B, None, C, None, D),        # a residual on a checkpoint
                 (None, cp, None, None, None, None, cp, B, C, D),       # from a checkpoint to one
                 (A, None, None, None, None, None, None, None, C, D),   # no out
                 (A, None, None, None, None, None, None, A, C, D),      # out over x
                 (A, None, None, B, None, None, None, B, C, D),         # out over weight
                 (A, None, None, None, None, None, None, B, C, C),      # mean over rstd
                 (A, None, B, None, None, C, None, C, None, D),         # x_out over out
                 (A, None, None, None, None, None, L.Checkpoint(B, G, 0), B, C, D),
                 (ctypes.c_void_p((1 << 20) + 1), None, None, None, None, None, None, B, C, D),
                 (ODD, None, None, None, None, None, cp, B, C, D)]:     # a checkpoint wants 16 bytes
        assert f(ok, *args, None) == L.ERR_INVALID_ARG, args
    assert f(L.Norm(4, 48, 0, 1e-5, 0, 0), A, None, None, None, None, None, cp, B, C, D,
             None) == L.ERR_INVALID_ARG
    assert f(L.Norm(4, 64, 0, 1e-5, 1, 0), ODD, None, None, None, None, None, None, B, C, D,
             None) == L.ERR_INVALID_ARG                                 # fp32 rows at 2 bytes
    assert f(ok, ODD, None, None, None, None, None, None, B, C, D, None) in reached
    assert f(ok, A, None, None, None, None, None, cp, B, C, D, None) in reached
    assert size(ok, None) == L.ERR_INVALID_ARG and size(ok, n) == 0 and n.value > 0
    #     d_out, x, from, mean, rstd, weight, g, dx, d_weight, d_bias, ws, bytes
    m = n.value
    for args in [(None, B, None, C, C, None, None, D, None, None, None, 0),
                 (A, None, None, C, C, None, None, D, None, None, None, 0),
                 (A, B, cp, C, C, None, None, D, None, None, None, 0),
                 (A, B, None, None, C, None, None, D, None, None, None, 0),   # layer without mean
                 (A, B, None, C, None, None, None, D, None, None, None, 0),
                 (A, B, None, C, C, None, None, None, None, None, None, 0),
                 (A, B, None, C, C, None, None, A, None, None, None, 0),      # dx over d_out
                 (A, B, None, C, C, None, None, B, None, None, None, 0),      # dx over x
                 (A, B, None, C, C, None, None, D, F, F, G, m),               # d_weight over d_bias
                 (A, B, None, C, C, None, None, D, F, None, None, m),         # no scratch
                 (A, B, None, C, C, None, None, D, F, None, D, m),            # scratch over dx
                 (A, B, None, C, C, None, None, D, F, None, ODD, m)]:
        assert b(ok, *args, None) == L.ERR_INVALID_ARG, args
    assert b(ok, A, B, None, C, C, None, None, D, F, None, G, m - 1, None) == L.ERR_WORKSPACE_TOO_SMALL
    assert b(ok, A, B, None, C, C, None, D, D, F, None, G, m, None) in reached  # dx may be g
    assert b(L.Norm(4, 64, 1, 1e-5, 0, 0), A, B, None, None, C, None, None, D, None, None, None, 0,
             None) in reached


def test_scratch_stays_bounded(L):
    from mxfp4_quantized_moe_b200 import moe
    assert moe.norm_workspace_bytes(0, 64) == 0
    assert moe.norm_workspace_bytes(1, 64) >= 8 * 64
    assert moe.norm_workspace_bytes(2 ** 31 - 1, 2880) <= 64 << 20


def test_wrappers_refuse_cpu_tensors_and_bad_names():
    from mxfp4_quantized_moe_b200 import moe
    with pytest.raises(ValueError):
        moe.route(moe.Routing(2), torch.zeros(3, 8))
    with pytest.raises(ValueError):
        moe.route(moe.Routing(2), torch.zeros(8))
    with pytest.raises(ValueError):
        moe.norm_forward(torch.zeros(3, 8))
    with pytest.raises(ValueError):
        moe.checkpoint_pack(torch.zeros(3, 32))
    with pytest.raises(ValueError):
        moe.Routing(2, "relu").dims(3, 8)
    with pytest.raises(ValueError):
        moe.norm_forward(torch.zeros(3, 8), kind="batch")
    with pytest.raises(TypeError):
        moe.norm_forward(torch.zeros(3, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        moe.Checkpoint.empty(3, 40, device="cpu")
    cp = moe.Checkpoint.empty(3, 64, device="cpu")
    with pytest.raises(ValueError):
        moe.norm_forward(cp, y=torch.zeros(3, 64))
    with pytest.raises(ValueError):
        moe.norm_forward(cp, checkpoint="int8")
    with pytest.raises(ValueError):
        moe.norm_forward(torch.zeros(3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.checkpoint_unpack(cp)


def test_grad_chain_without_dx(L, reached):
    gc = L.lib.mxfp4_moe_grad_chain
    assert gc(4, 64, 8, A, None, B, C, D, None) in reached
    assert gc(4, 64, 8, A, ODD, B, C, D, None) == L.ERR_INVALID_ARG


def test_the_one_step_binding_leaves_other_calls_to_the_wrappers():
    """_edge answers None, with no error set, for whatever is not a plain call."""
    from mxfp4_quantized_moe_b200 import moe
    e = moe._edge
    x, l = torch.zeros(3, 64), torch.zeros(3, 8)
    how = (2, "softmax", 1, 1, 1, True, 1.0)
    idx = torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: e.route(*how, l, None), lambda: e.route(*how, None, None),
                 lambda: e.route("two", *how[1:], l, None), lambda: e.route(*how, 7, "b"),
                 lambda: e.route(2, "relu", *how[2:], l, None),
                 lambda: e.route_backward(*how, l, idx, torch.zeros(3, 2), torch.zeros(3, 2)),
                 lambda: e.norm_forward(x, None, None, False, None, None, None, "layer", 1e-5, None),
                 lambda: e.norm_forward(x, x, "e4m3", False, None, None, None, "rms", "eps", None),
                 lambda: e.norm_backward(x, x, None, None, None, x, None, "rms", None),
                 lambda: e.checkpoint_pack(x, "e4m3"), lambda: e.checkpoint_pack(x, 3),
                 lambda: e.checkpoint_unpack(x, None, "e4m3", False)):
        assert call() is None
    with pytest.raises(TypeError):
        e.route(l)
