"""The norm, its gradients and 8-bit checkpoints on the GPU against the fp64 oracle.

Bounds, with r = 2^-24 (half a step of fp32) and u the half step of the rows' type: a row's sums
run over at most 32 features a thread and ten levels of shuffles, so 64 r covers each, relative
to the sum of magnitudes.  They follow each formula's terms; nothing is fitted.
"""

import numpy as np
import pytest
import torch

from oracle import edge_oracle as O

pytestmark = pytest.mark.gpu
R = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mxfp4_quantized_moe_b200 import moe as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(T, H, dtype, seed, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, generator=g) * scale + offset).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def hat_bound(x, mean, rstd, kind):
    """How far x_hat may be off: the mean's sum, the subtraction, and rstd."""
    m = np.abs(x).mean(1, keepdims=True)
    e_mean = 64 * R * m if kind == "layer" else 0.0
    rel = 64 * R + (e_mean * rstd[:, None]) ** 2
    hat = (x - mean[:, None]) * rstd[:, None]
    return rstd[:, None] * (e_mean + R * (np.abs(x) + m)) + np.abs(hat) * (rel + 4 * R)


def check_forward(out, mean, rstd, x, w, b, kind, dtype, eps=1e-5):
    ref, rm, rr = O.norm(x, w, b, kind, eps)
    wa = 1.0 if w is None else np.abs(w)
    ba = 0.0 if b is None else np.abs(b)
    hat = np.abs((x - rm[:, None]) * rr[:, None])
    tol = hat_bound(x, rm, rr, kind) * wa + 4 * R * (hat * wa + ba)
    tol = tol + half_step(dtype) * (np.abs(ref) + tol) + 1e-38
    assert np.all(np.abs(f64(out) - ref) <= tol), (np.abs(f64(out) - ref) / tol).max()
    m = np.abs(x).mean(1)
    if kind == "layer":
        assert np.all(np.abs(f64(mean) - rm) <= 64 * R * m + 1e-38)
    assert np.all(np.abs(f64(rstd) - rr) <= rr * (64 * R + (64 * R * m * rr) ** 2))


def check_backward(dx, dw, db, d_out, x, w, kind, dtype, g=None, eps=1e-5):
    rx, rw, rb = O.norm_backward(d_out, x, w, kind, eps, g)
    hat, rm, rr = O.norm(x, kind=kind, eps=eps)
    wa = np.ones(x.shape[1]) if w is None else w
    v = np.abs(d_out * wa)
    eh = hat_bound(x, rm, rr, kind)
    mean = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    c2 = mean(v * np.abs(hat))
    e_c2 = mean(v * eh) + 68 * R * c2
    inner = v + np.abs(hat) * c2
    e = 4 * R * inner + np.abs(hat) * e_c2 + eh * c2
    if kind == "layer":
        e = e + 68 * R * mean(v)
        inner = inner + mean(v)
    rel = 68 * R + (64 * R * mean(np.abs(x)) * rr[:, None]) ** 2
    tol = rr[:, None] * (e + rel * inner)
    if g is not None:
        tol = tol + 2 * R * (np.abs(g) + rr[:, None] * inner)
    tol = tol + half_step(dtype) * (np.abs(rx) + tol) + 1e-38
    assert np.all(np.abs(f64(dx) - rx) <= tol), (np.abs(f64(dx) - rx) / tol).max()
    steps = len(x) / 148 + 64  # rows in sequence of a thread, then the parts
    if dw is not None:
        tol = (np.abs(d_out) * eh).sum(0) + steps * R * np.abs(d_out * hat).sum(0) + 1e-38
        assert np.all(np.abs(f64(dw) - rw) <= tol), (np.abs(f64(dw) - rw) / tol).max()
    if db is not None:
        tol = steps * R * np.abs(d_out).sum(0) + 1e-38
        assert np.all(np.abs(f64(db) - rb) <= tol)


SHAPES = [(1, 1), (1, 2880), (3, 7), (5, 33), (2, 64), (17, 96), (700, 256), (9, 1000), (4, 1001),
          (300, 2880), (1203, 520), (3, 4096), (2, 8192), (3, 12000), (5, 16384), (2, 16383),
          # many rows: the persistent forms, of whole vectors and of any length
          (1301, 32), (1500, 2880), (620, 4096), (601, 8192), (600, 16384), (2000, 1), (1400, 7),
          (650, 61), (900, 255), (610, 1001), (640, 2879), (603, 4099), (601, 7001), (600, 12001)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm(moe, T, H, dtype, kind):
    """Forward and backward; parameters of the other type; with and without residual and g."""
    dt, pt = TYPES[dtype], TYPES["fp32" if dtype == "bf16" else "bf16"]
    x = rows(T, H, dt, T + H, 3.0, 0.5)
    y, d, g = rows(T, H, dt, 1), rows(T, H, dt, 2), rows(T, H, dt, 3)
    w = rows(1, H, pt, 4, 0.3, 1.0)[0]
    b = rows(1, H, pt, 5, 0.3)[0] if kind == "layer" else None
    xs = (x.float() + y.float()).to(dt)
    f = moe.norm_forward(x.cuda(), w.cuda(), None if b is None else b.cuda(), kind=kind,
                         y=y.cuda())
    assert torch.equal(f.x_out.cpu(), xs)
    assert (f.mean is None) == (kind == "rms") and f.checkpoint is None
    wn, bn = f64(w), None if b is None else f64(b)
    check_forward(f.out, f.mean, f.rstd, f64(xs), wn, bn, kind, dt)
    dx, dw, db = moe.norm_backward(d.cuda(), f.x_out, f.mean, f.rstd, w.cuda(), kind=kind,
                                   g=g.cuda())
    assert (db is None) == (kind == "rms")
    check_backward(dx, dw, db, f64(d), f64(xs), wn, kind, dt, f64(g))
    # no residual, no parameters, no gradient of theirs
    f = moe.norm_forward(x.cuda(), kind=kind)
    check_forward(f.out, f.mean, f.rstd, f64(x), None, None, kind, dt)
    dx, dw, db = moe.norm_backward(d.cuda(), x.cuda(), f.mean, f.rstd, kind=kind, params=False)
    assert dw is None and db is None
    check_backward(dx, None, None, f64(d), f64(x), None, kind, dt)


@pytest.mark.parametrize("format", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (65, 256), (7, 2880), (2, 8192), (1, 16384)])
def test_checkpoint(moe, T, H, dtype, format):
    """Codes, scale bytes and values bit for bit, over magnitudes from subnormal to the largest,
    and blocks with an infinity or NaN."""
    dt = TYPES[dtype]
    x = rows(T, H, torch.float32, H, 1.0)
    gen = torch.Generator().manual_seed(6)
    x = x * torch.exp2(torch.randint(-140, 127, (T, H // 32), generator=gen).float()
                       ).repeat_interleave(32, 1)
    x[0, :32] = 0.0
    x[0, 1] = -0.0
    if T > 1:
        x[1, 33], x[1, 64], x[T - 1, 5] = float("inf"), float("nan"), torch.finfo(dt).max
    x = x.to(dt)
    codes, scales, values = O.checkpoint(f64(x), format)
    cp = moe.checkpoint_pack(x.cuda(), format)
    assert np.array_equal(cp.scales.cpu().numpy(), scales)
    live = np.repeat(scales != 255, 32, axis=1)
    assert np.array_equal(cp.codes.cpu().numpy()[live], codes[live])
    for out in (torch.float32, torch.bfloat16):
        got = moe.checkpoint_unpack(cp, out).cpu()
        ref = torch.from_numpy(values).float().to(out)
        assert torch.equal(torch.isnan(got), torch.from_numpy(~live))
        assert torch.equal(got[torch.from_numpy(live)], ref[torch.from_numpy(live)])
        assert torch.isfinite(got[torch.from_numpy(live)]).all()


def test_unpack_reads_every_scale_byte(moe):
    """Scale bytes 0 to 254 as 2^(byte - 127), 255 as NaN, with every code."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 8)
    for format in ("e4m3", "int8"):
        cp = moe.Checkpoint(codes.cuda(), scales.cuda(), format)
        got = moe.checkpoint_unpack(cp, torch.float32).cpu()
        if format == "e4m3":
            v = codes.view(torch.float8_e4m3fn).double()
        else:
            v = codes.view(torch.int8).double() / 64
        ref = (v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)).float()
        ref[255] = float("nan")
        assert torch.equal(torch.nan_to_num(got, nan=1.5), torch.nan_to_num(ref, nan=1.5))


@pytest.mark.parametrize("format", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", [(1, 32), (5, 96), (130, 256), (300, 2880), (3, 16384)])
def test_norm_beside_and_from_a_checkpoint(moe, T, H, kind, dtype, format):
    """The checkpoint that the norm's forward fills is that of its rows, and the norm and its
    gradients from a checkpoint are those of the rows it stands for."""
    dt = TYPES[dtype]
    x, y, d, g = (rows(T, H, dt, s, 2.0) for s in range(4))
    w = rows(1, H, dt, 4, 0.3, 1.0)[0]
    xs = (x.float() + y.float()).to(dt)
    f = moe.norm_forward(x.cuda(), w.cuda(), kind=kind, y=y.cuda(), checkpoint=format)
    plain = moe.norm_forward(x.cuda(), w.cuda(), kind=kind, y=y.cuda())
    alone = moe.checkpoint_pack(xs.cuda(), format)
    assert torch.equal(f.out, plain.out) and torch.equal(f.x_out.cpu(), xs)
    assert torch.equal(f.checkpoint.codes, alone.codes)
    assert torch.equal(f.checkpoint.scales, alone.scales)
    kept = moe.norm_forward(x.cuda(), w.cuda(), kind=kind, checkpoint=format)  # no residual
    again = moe.checkpoint_pack(x.cuda(), format)
    assert torch.equal(kept.checkpoint.codes, again.codes)
    assert torch.equal(kept.checkpoint.scales, again.scales)

    v = f64(moe.checkpoint_unpack(alone, torch.float32))
    n = moe.norm_forward(alone, w.cuda(), kind=kind, dtype=dt)
    check_forward(n.out, n.mean, n.rstd, v, f64(w), None, kind, dt)
    dx, dw, db = moe.norm_backward(d.cuda(), alone, n.mean, n.rstd, w.cuda(), kind=kind,
                                   g=g.cuda())
    check_backward(dx, dw, db, f64(d), v, f64(w), kind, dt, f64(g))


def test_rows_far_from_zero(moe):
    """A mean a thousand times the spread: the variance is taken about the mean."""
    x = rows(6, 2880, torch.float32, 1, 1.0, 1000.0)
    f = moe.norm_forward(x.cuda())
    check_forward(f.out, f.mean, f.rstd, f64(x), None, None, "layer", torch.float32)
    ref = O.norm(f64(x))[0]
    assert np.abs(f64(f.out) - ref).max() < 2e-2


def test_a_bad_row_stays_alone(moe):
    x = rows(9, 96, torch.bfloat16, 1)
    clean = moe.norm_forward(x.cuda())
    bad = x.clone()
    bad[3, 5], bad[6, 0] = float("nan"), float("inf")
    f = moe.norm_forward(bad.cuda())
    ok = torch.tensor([t not in (3, 6) for t in range(9)])
    assert torch.equal(f.out.cpu()[ok], clean.out.cpu()[ok])
    assert torch.isnan(f.out.cpu()[~ok]).any(1).all()
    # constant rows: variance 0, out = bias
    c = torch.full((2, 96), 3.0, dtype=torch.bfloat16, device="cuda")
    b = torch.arange(96, device="cuda").float()
    assert torch.equal(moe.norm_forward(c, None, b).out, b.bfloat16().expand(2, 96))


def test_in_place_gradient_and_outputs_of_the_caller(moe):
    T, H = 21, 288
    x, d, g = (rows(T, H, torch.bfloat16, s).cuda() for s in range(3))
    w = rows(1, H, torch.bfloat16, 4, 0.3, 1.0)[0].cuda()
    f = moe.norm_forward(x, w)
    dx, dw, db = moe.norm_backward(d, x, f.mean, f.rstd, w, g=g)
    g2 = g.clone()
    ws = torch.empty(moe.norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
    got = moe.norm_backward(d, x, f.mean, f.rstd, w, g=g2, dx=g2, d_weight=dw2, d_bias=db2, ws=ws)
    assert got[0] is g2 and got[1] is dw2 and got[2] is db2
    assert torch.equal(g2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    # rows behind the last one stay as they were
    out = torch.full((T + 2, H), 9.0, dtype=torch.bfloat16, device="cuda")
    cp = moe.Checkpoint(torch.full((T + 2, H), 77, dtype=torch.uint8, device="cuda"),
                        torch.full((T + 2, H // 32), 77, dtype=torch.uint8, device="cuda"), "int8")
    head = moe.Checkpoint(cp.codes[:T], cp.scales[:T], "int8")
    moe.norm_forward(x, w, out=out[:T], checkpoint=head)
    assert torch.equal(out[:T], f.out) and (out[T:] == 9).all()
    assert (cp.codes[T:] == 77).all() and (cp.scales[T:] == 77).all()
    out.fill_(9.0)
    moe.norm_backward(d, x, f.mean, f.rstd, w, g=g, dx=out[:T])
    assert torch.equal(out[:T], dx) and (out[T:] == 9).all()


@pytest.mark.parametrize("T", [19, 700])
@pytest.mark.parametrize("H", [64, 61, 512])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_without_vector_alignment(moe, H, dtype, T):
    """Views that begin at any element give the same values as aligned copies."""
    dt = TYPES[dtype]
    base = [rows(1, T * H + 8, dt, s)[0].cuda() for s in range(4)]
    for off in (1, 2, 4):
        x, y, d, g = (t[off:off + T * H].view(T, H) for t in base)
        w = base[0][off:off + H]
        f = moe.norm_forward(x, w, y=y)
        a = moe.norm_forward(x.clone(), w.clone(), y=y.clone())
        check_forward(f.out, f.mean, f.rstd, f64(a.x_out), f64(w), None, "layer", dt)
        assert torch.equal(f.x_out, a.x_out)
        dx, dw, db = moe.norm_backward(d, f.x_out, f.mean, f.rstd, w, g=g)
        check_backward(dx, dw, db, f64(d), f64(a.x_out), f64(w), "layer", dt, f64(g))


@pytest.mark.parametrize("T", [1, 2, 5, 400])
def test_parameter_gradients_at_any_address(moe, T):
    """Outputs of the parameters' gradients that begin at any fp32 element."""
    H = 320
    x, d = rows(T, H, torch.bfloat16, 1).cuda(), rows(T, H, torch.bfloat16, 2).cuda()
    f = moe.norm_forward(x)
    _, dw, db = moe.norm_backward(d, x, f.mean, f.rstd)
    base = torch.full((2, H + 4), 5.0, device="cuda")
    for off in (1, 2, 3):
        a, b = base[0, off:off + H], base[1, off:off + H]
        moe.norm_backward(d, x, f.mean, f.rstd, d_weight=a, d_bias=b)
        assert torch.equal(a, dw) and torch.equal(b, db)
        assert base[:, :1].eq(5).all()
        cp = moe.checkpoint_pack(x)
        n = moe.norm_forward(cp)
        moe.norm_backward(d, cp, n.mean, n.rstd, d_weight=a, d_bias=b)
        assert torch.isfinite(a).all() and torch.equal(b, db)


@pytest.mark.parametrize("H", [8192, 8189])
def test_rows_past_32_bit_offsets(moe, H):
    """Rows of more than 2^31 elements: the last ones as in a batch of their own."""
    T, n = 2 ** 31 // H + 700, 650
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_()
    tail = x[-n:].clone()
    f, t = moe.norm_forward(x), moe.norm_forward(tail)
    assert torch.equal(f.out[-n:], t.out) and torch.equal(f.rstd[-n:], t.rstd)
    dx, _, _ = moe.norm_backward(f.out, x, f.mean, f.rstd)
    dt, _, _ = moe.norm_backward(t.out, tail, t.mean, t.rstd)
    assert torch.equal(dx[-n:], dt)
    if H % 32 == 0:
        cp = moe.checkpoint_pack(x, "int8")
        ct = moe.checkpoint_pack(tail, "int8")
        assert torch.equal(cp.codes[-n:], ct.codes) and torch.equal(cp.scales[-n:], ct.scales)
        assert torch.equal(moe.checkpoint_unpack(cp)[-n:], moe.checkpoint_unpack(ct))
        again = moe.norm_forward(cp)
        assert torch.equal(again.out[-n:], moe.norm_forward(ct).out)


def test_empty_batch(moe):
    for dt in TYPES.values():
        x = torch.empty(0, 64, dtype=dt, device="cuda")
        f = moe.norm_forward(x, y=x, checkpoint="e4m3")
        assert f.out.shape == f.x_out.shape == (0, 64) and f.checkpoint.scales.shape == (0, 2)
        dw = torch.ones(64, device="cuda")
        dx, dw, db = moe.norm_backward(x, x, f.mean, f.rstd, d_weight=dw)
        assert dx.shape == (0, 64) and not dw.any() and not db.any()
        assert moe.checkpoint_unpack(moe.checkpoint_pack(x), dt).shape == (0, 64)


def test_same_bits_every_time_on_any_stream_and_in_a_graph(moe):
    T, H = 1500, 2880
    x, y, d = (rows(T, H, torch.bfloat16, s).cuda() for s in range(3))
    w, b = rows(1, H, torch.bfloat16, 4)[0].cuda(), rows(1, H, torch.bfloat16, 5)[0].cuda()

    def step(x, stream=None):
        f = moe.norm_forward(x, w, b, y=y, checkpoint="e4m3", stream=stream)
        n = moe.norm_forward(f.checkpoint, w, b, stream=stream)
        return (f.out, f.x_out, n.out) + moe.norm_backward(d, f.checkpoint, n.mean, n.rstd, w,
                                                            g=y, stream=stream)
    first = step(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = step(x, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    static = x.clone()
    with torch.cuda.graph(graph):
        held = step(static)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, o, h in zip(first, other, held):
        assert torch.equal(a, o) and torch.equal(a, h)
    static.copy_(d)
    graph.replay()
    for a, h in zip(step(static), held):
        assert torch.equal(a, h)
