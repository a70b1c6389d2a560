"""Corners of the operators at the block's edge on the GPU: calls that the documentation allows
and that ordinary batches do not reach, against the fp64 oracle or the entry points themselves.
"""

import threading

import numpy as np
import pytest
import torch

from oracle import edge_oracle as O

from test_gpu_norm import R, TYPES, check_backward, check_forward, f64, hat_bound, rows
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


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,k", [(8, 4, 2), (32, 4, 2), (64, 4, 4), (128, 8, 4), (40, 5, 1)])
def test_group_sums_below_the_lowest_value(moe, E, groups, k, scores):
    """Two keys may sum to less than fp32 holds: such a group still comes before one that has no
    expert left, and after all others."""
    logits = normal(40, E, E + 2)
    size = E // groups
    logits.view(-1, groups, size)[:, 0] = float("-inf")
    logits.view(-1, groups, size)[::4, 3, 1:] = float("-inf")
    low = torch.finfo(torch.float32).min
    for level in (0.75 * low, 0.5 * low):
        bias = normal(1, E, 43, 0.05)[0].view(groups, size)
        bias[1:3] = level
        for top_groups in range(1, groups + 1):
            if top_groups * size >= k:
                r = moe.Routing(k, scores, groups, top_groups, 2, renormalize=False)
                check(moe, r, logits, bias.reshape(E))


# ---- host threads ---------------------------------------------------------------------------
def test_first_call_of_a_host_thread(moe):
    """The library's calls take up the device's context in a host thread that has made no CUDA
    call yet, the ones that describe their operands to the driver first among them."""
    from mxfp4_quantized_moe_b200 import inputs
    L = moe._lib
    T, H, I, E, k = 40, 64, 64, 4, 2
    inp = inputs.make_layer(T, H, I, E, k, 9)
    shape, w = moe.MoeShape(T, H, I, E, k), moe.weights_to(inp, "cuda")
    ws, wt = moe.alloc_workspace(shape), moe.transpose_weights(shape, w)
    x, dy = inp["x"].cuda(), inp["dy"].cuda()
    lg = inp["logits"].cuda()
    off = torch.tensor([0, 5, 20, 20, 40], dtype=torch.int32).cuda()
    y = moe.forward(shape, w, x, lg, ws)
    dx, dw, dl = moe.backward_input(shape, w, wt, dy, ws)
    p = moe.grouped_matmul(off, x, w["gu_blocks"], w["gu_scales"], 2 * I)
    moe.forward(shape, w, x, lg, ws)  # the state that the backward used up
    outs = [torch.empty_like(t) for t in (y, dx, dw, dl, p)]
    yp, dxp, dwp, dlp, pp = (t.data_ptr() for t in outs)
    dims, weights = shape.dims(), moe._weights(w)
    calls = {
        "grouped_matmul": (E, 2 * I, H, T, off.data_ptr(), x.data_ptr(), w["gu_blocks"].data_ptr(),
                           w["gu_scales"].data_ptr(), 0, pp, None, None),
        "backward_input": (dims, weights, wt.data_ptr(), wt.numel(), dy.data_ptr(), ws.data_ptr(),
                           ws.numel(), dxp, dwp, dlp, None),
        "forward": (dims, weights, x.data_ptr(), lg.data_ptr(), yp, None, None, ws.data_ptr(),
                    ws.numel(), None),
    }
    torch.cuda.synchronize()
    for name, args in calls.items():
        got = []
        t = threading.Thread(target=lambda: got.append(getattr(L.lib, "mxfp4_moe_" + name)(*args)))
        t.start()
        t.join()
        assert got == [L.OK], name
    torch.cuda.synchronize()
    for a, b in zip(outs, (y, dx, dw, dl, p)):
        assert torch.equal(a, b)


def run_at_once(*calls, times=300):
    """Each call many times over in a host thread of its own, on a stream of its own."""
    errors, start = [], threading.Barrier(len(calls))

    def loop(call):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(times):
                call(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 (shown by the assertion)
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:3]


@pytest.mark.parametrize("dtype,T,lengths", [
    ("bf16", 640, (2304, 2880)), ("bf16", 640, (2305, 2881)), ("fp32", 640, (3400, 4096)),
    ("fp32", 640, (4200, 8184)), ("bf16", 640, (4200, 8191))])
def test_norm_of_two_lengths_in_two_threads(moe, dtype, T, lengths):
    """Rows of different lengths that share a kernel, from two host threads at once: the library's
    calls alone, one after another, which let the other thread run."""
    L, dt = moe._lib, TYPES[dtype]
    fmt = L.ROWS_FP32 if dtype == "fp32" else L.ROWS_BF16

    def call(H):
        x, y, d = (rows(T, H, dt, s).cuda() for s in range(3))
        w = rows(1, H, dt, 4, 0.3, 1.0)[0].cuda()
        f = moe.norm_forward(x, w, y=y)
        dx, dw, db = moe.norm_backward(d, f.x_out, f.mean, f.rstd, w, g=y)
        out, xo, mean, rstd, gx, gw, gb = (torch.empty_like(t) for t in (
            f.out, f.x_out, f.mean, f.rstd, dx, dw, db))
        ws = torch.empty(moe.norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        p = [t.data_ptr() for t in (x, y, w, xo, out, mean, rstd, d, gx, gw, gb, ws)]
        x_, y_, w_, xo_, out_, mean_, rstd_, d_, gx_, gw_, gb_, ws_ = p
        dims, n = L.Norm(T, H, L.NORMS["layer"], 1e-5, fmt, fmt), ws.numel()

        def once(stream):
            s = stream.cuda_stream
            L.check(L.lib.mxfp4_moe_norm_forward(dims, x_, None, y_, w_, None, xo_, None, out_,
                                                 mean_, rstd_, s), "forward")
            L.check(L.lib.mxfp4_moe_norm_backward(dims, d_, xo_, None, mean_, rstd_, w_, y_, gx_,
                                                  gw_, gb_, ws_, n, s), "backward")

        def same():
            for a, b in ((out, f.out), (gx, dx), (gw, dw), (gb, db)):
                assert torch.equal(a, b)
            return x, y, w, d, ws, xo, mean, rstd  # alive until here
        return once, same

    pairs = [call(H) for H in lengths]
    torch.cuda.synchronize()
    run_at_once(*(p[0] for p in pairs), times=4000)
    for _, same in pairs:
        same()


def test_products_and_gradient_chains_in_two_threads(moe):
    """The experts' product with two K, and the gradient chain with two E, from two host threads:
    the launches of one leave the other's limits alone."""
    L, gen = moe._lib, torch.Generator().manual_seed(5)
    off = torch.tensor([0, 20, 64], dtype=torch.int32).cuda()

    def product(K, E):
        x = torch.randn(64, K, generator=gen).bfloat16().cuda()
        blocks = torch.randint(0, 256, (2, 64, K // 2), generator=gen, dtype=torch.uint8).cuda()
        scales = torch.randint(120, 130, (2, 64, K // 32), generator=gen, dtype=torch.uint8).cuda()
        g = torch.randn(64, 256, generator=gen).bfloat16().cuda()
        dl = torch.randn(64, E, generator=gen).cuda()
        w_r = torch.randn(256, E, generator=gen).bfloat16().cuda()
        want = moe.grouped_matmul(off, x, blocks, scales, 64), moe.grad_chain(g, None, dl, w_r)
        out = [torch.empty_like(t) for t in want]
        held = (off, x, blocks, scales, g, dl, w_r, *out)
        off_, x_, blocks_, scales_, g_, dl_, w_, out_, chain_ = (t.data_ptr() for t in held)

        def once(stream):
            s = stream.cuda_stream
            L.check(L.lib.mxfp4_moe_grouped_matmul(2, 64, K, 64, off_, x_, blocks_, scales_, 0, out_,
                                                   None, s), "product")
            L.check(L.lib.mxfp4_moe_grad_chain(64, 256, E, g_, None, dl_, w_, chain_, s), "chain")

        def same():
            assert all(torch.equal(a, b) for a, b in zip(held[-2:], want))
        return once, same

    pairs = [product(128, 16), product(2880, 256)]
    torch.cuda.synchronize()
    run_at_once(*(p[0] for p in pairs), times=4000)
    for _, same in pairs:
        same()


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


# ---- autograd forms -------------------------------------------------------------------------
@pytest.mark.parametrize("format", ["e4m3", "int8"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd_norm_from_a_checkpoint_is_the_gradient_at_its_rows(moe, kind, format, dtype):
    """The forward is that of the exact rows; the backward is the norm's gradient at the rows that
    the checkpoint stands for, statistics included."""
    from mxfp4_quantized_moe_b200.autograd import norm
    T, H, dt = 70, 96, TYPES[dtype]
    x, y, d, g = (rows(T, H, dt, s, 2.0, 0.5) for s in range(4))
    w = rows(1, H, dt, 4, 0.3, 1.0)[0]
    for residual in (False, True):
        leaves = [t.cuda().requires_grad_(True) for t in ((x, w, y) if residual else (x, w))]
        out = norm(leaves[0], leaves[1], residual=leaves[2] if residual else None, kind=kind,
                   checkpoint=format)
        n, xs = out if residual else (out, leaves[0])
        ref = moe.norm_forward(xs.detach(), leaves[1].detach(), kind=kind)
        assert torch.equal(n, ref.out)
        torch.autograd.backward([n, xs] if residual else [n],
                                [d.cuda(), g.cuda()] if residual else [d.cuda()])
        _, _, v = O.checkpoint(f64(xs), format)
        check_backward(leaves[0].grad, None, None, f64(d), v, f64(w), kind, dt,
                       f64(g) if residual else None)
        hat, mean, rstd = O.norm(v, kind=kind)
        want = (f64(d) * hat).sum(0)
        # 70 rows in sequence at most; then one rounding to the parameter's type
        tol = (np.abs(f64(d)) * hat_bound(v, mean, rstd, kind)).sum(0)
        tol = tol + 72 * R * np.abs(f64(d) * hat).sum(0)
        tol = tol + torch.finfo(dt).eps / 2 * (np.abs(want) + tol)
        assert np.all(np.abs(f64(leaves[1].grad) - want) <= tol)
        if residual:
            assert torch.equal(leaves[2].grad, leaves[0].grad)



def test_saved_tensor_hooks_see_all_that_is_kept(moe):
    """Offloading what the graph keeps takes the checkpoint's scales along with its codes."""
    from mxfp4_quantized_moe_b200.autograd import norm
    x = rows(6, 64, torch.bfloat16, 1).cuda().requires_grad_(True)
    seen = []

    def pack(t):
        seen.append((tuple(t.shape), t.dtype))
        return t.cpu()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.cuda()):
        out = norm(x, checkpoint="int8")
    assert ((6, 64), torch.uint8) in seen and ((6, 2), torch.uint8) in seen
    assert not any(isinstance(v, torch.Tensor) for v in vars(out.grad_fn).values())
    out.backward(torch.ones_like(out))
    first, x.grad = x.grad, None
    norm(x, checkpoint="int8").backward(torch.ones_like(out))
    assert torch.equal(first, x.grad)


@pytest.mark.parametrize("shape", [(6, 64), (2, 3, 64), (0, 64)])
@pytest.mark.parametrize("checkpoint", [None, "e4m3"])
def test_autograd_outputs_may_be_changed_in_place(moe, shape, checkpoint):
    """As torch's own norms allow; a stream that the backward still reads is refused there."""
    from mxfp4_quantized_moe_b200.autograd import norm
    x = torch.randn(shape, device="cuda", requires_grad=True)
    y = torch.randn(shape, device="cuda", requires_grad=True)
    d = torch.randn(shape, device="cuda")

    def grads(change):
        x.grad = y.grad = None
        n = norm(x, checkpoint=checkpoint)
        n = n.mul_(2.0) if change else n * 2.0
        m, s = norm(x, residual=y, checkpoint=checkpoint)
        m = m.add_(1.0) if change else m + 1.0
        assert n.shape == m.shape == s.shape == shape
        (n + m * 3.0).backward(d)
        return x.grad, y.grad

    for a, b in zip(grads(True), grads(False)):
        assert torch.equal(a, b)
    m, s = norm(x, residual=y, checkpoint=checkpoint)
    s.mul_(2.0)
    if checkpoint:  # the rows are kept in 8 bits, the stream itself is free
        (m + s).sum().backward()
    else:
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            (m + s).sum().backward()


# ---- checkpoints beside tensors without 16-byte alignment -----------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_inputs_at_any_address_with_a_checkpoint(moe, dtype):
    """Rows and parameters that are slices of larger buffers, wherever they begin."""
    from mxfp4_quantized_moe_b200.autograd import norm
    T, H, dt = 5, 96, TYPES[dtype]

    def at(t, off):  # a copy that begins off elements behind an aligned address
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
        buf[off:].copy_(t.reshape(-1))
        return buf[off:].view(t.shape)

    base = [rows(T, H, dt, s).cuda() for s in range(4)]
    params = [rows(1, H, dt, s, 0.3, 1.0)[0].cuda() for s in (4, 5)]
    x, y, d, g = base
    f = moe.norm_forward(x, *params, y=y, checkpoint="int8")
    n = moe.norm_forward(f.checkpoint, *params, dtype=dt)
    b = moe.norm_backward(d, f.checkpoint, n.mean, n.rstd, params[0], g=g)
    for off in (1, 3):
        (xo, yo, do, go), po = [at(t, off) for t in base], [at(t, off) for t in params]
        assert xo.data_ptr() % 16
        f2 = moe.norm_forward(xo, *po, y=yo, checkpoint="int8")
        n2 = moe.norm_forward(f2.checkpoint, *po, dtype=dt)
        b2 = moe.norm_backward(do, f2.checkpoint, n2.mean, n2.rstd, po[0], g=go)
        for p, q in ((f.out, f2.out), (f.x_out, f2.x_out), (f.checkpoint.codes, f2.checkpoint.codes),
                     (f.checkpoint.scales, f2.checkpoint.scales), (n.out, n2.out), *zip(b, b2)):
            assert torch.equal(p, q)
        assert torch.equal(moe.checkpoint_pack(xo, "e4m3").codes, moe.checkpoint_pack(x, "e4m3").codes)
        xl, wl = xo.detach().requires_grad_(True), po[0].detach().requires_grad_(True)
        out = norm(xl, wl, po[1], residual=yo, checkpoint="int8")
        torch.autograd.backward(out, [do, go])
        assert torch.equal(out[0], f.out) and torch.equal(xl.grad, b[0])
        # the gradient added in place stays in place
        g3 = at(g, off)
        with pytest.raises(moe._lib.MoeError):
            moe.norm_backward(do, f.checkpoint, n.mean, n.rstd, params[0], g=g3, dx=g3)
        # outputs of the caller are not copied: refused as before
        with pytest.raises(moe._lib.MoeError):
            moe.norm_forward(x, out=xo, checkpoint="int8")


# ---- many rows with checkpoints -------------------------------------------------------------
def stored(x, format):
    """Codes, scale bytes and values of finite rows by the definition, block by block of 32."""
    b = x.double().view(x.shape[0], -1, 32)
    limit, bias = (448.0, 127) if format == "e4m3" else (127.0, 133)
    most = b.abs().amax(2, keepdim=True)
    m, e = torch.frexp(most / limit)
    S = torch.where(m > 0.5, e, e - 1)  # the least S with most <= limit 2^S
    S = torch.where(most > 0, S, -126).clamp(min=-126)
    v = torch.ldexp(b, -S)
    if format == "e4m3":
        v = v.float().to(torch.float8_e4m3fn)
        codes, v = v.view(torch.uint8), v.double()
    else:
        v = v.round()
        codes = v.to(torch.int8).view(torch.uint8)
    return (codes.view(x.shape), (S + bias).to(torch.uint8).view(x.shape[0], -1),
            torch.ldexp(v, S).view(x.shape))


@pytest.mark.parametrize("format", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,kind", [("bf16", "layer"), ("fp32", "rms")])
@pytest.mark.parametrize("T,H", [(601, 32), (15003, 96), (15003, 256), (4001, 1056), (1501, 2880),
                                 (1301, 4096), (623, 6144), (611, 8192), (603, 16384)])
def test_many_rows_beside_and_from_a_checkpoint(moe, T, H, kind, dtype, format):
    """Batches of several turns of the persistent forms, the last one ragged: the checkpoint that
    the forward fills, the norm from it, and the gradients from it."""
    dt = TYPES[dtype]
    x, y, d, g = (rows(T, H, dt, s, 2.0).cuda() for s in range(4))
    # magnitudes differ from block to block, so that no block's scale serves its neighbour
    x *= torch.exp2((torch.arange(H, device="cuda") // 32 % 5).to(dt))
    x *= torch.exp2((torch.arange(T, device="cuda") % 7).to(dt))[:, None]
    w = rows(1, H, dt, 4, 0.3, 1.0)[0].cuda()
    xs = (x.float() + y.float()).to(dt)
    f = moe.norm_forward(x, w, kind=kind, y=y, checkpoint=format)
    codes, scales, values = stored(xs.cpu(), format)
    assert torch.equal(f.x_out, xs)
    assert torch.equal(f.checkpoint.codes.cpu(), codes)
    assert torch.equal(f.checkpoint.scales.cpu(), scales)
    check_forward(f.out, f.mean, f.rstd, f64(xs), f64(w), None, kind, dt)
    kept = moe.norm_forward(xs, w, kind=kind, checkpoint=format)  # no residual
    assert torch.equal(kept.checkpoint.codes.cpu(), codes) and torch.equal(kept.out, f.out)
    assert torch.equal(kept.checkpoint.scales.cpu(), scales)
    v = values.numpy()
    n = moe.norm_forward(f.checkpoint, w, kind=kind, dtype=dt)
    check_forward(n.out, n.mean, n.rstd, v, f64(w), None, kind, dt)
    dx, dw, db = moe.norm_backward(d, f.checkpoint, n.mean, n.rstd, w, kind=kind, g=g)
    check_backward(dx, dw, db, f64(d), v, f64(w), kind, dt, f64(g))
    dx, _, _ = moe.norm_backward(d, f.checkpoint, n.mean, n.rstd, w, kind=kind)
    check_backward(dx, None, None, f64(d), v, f64(w), kind, dt)
