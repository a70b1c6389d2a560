"""Achieved HBM bandwidth of the memory-bound stages on one GPU.

    python -m mxfp4_quantized_moe_b200.kernel_bench [--iters N]

* standalone dequantization (`mxfp4_moe_dequantize`) of a whole gpt-oss-20b gate_up weight
  set, E*2I rows of H elements: 0.5 B of codes + 1/32 B of scale read and 2 B of bf16 written
  per element;
* the memory-bound kernels of one gpt-oss-20b layer step at T=8192, from the library's
  per-kernel event timing: the forward gather (`gather_x`: A rows of H bf16 read and
  written), the combines
  (`combine_y`, `combine_dx`: A rows read, T rows written) and the dY gather with the
  routing-weight dot (`gather_dy_dw`: A rows of dY and of y read, A rows written);
* the operators at the block's edge at the stack's size, T=32768, H=2880 (each through its own
  entry point): the norm's forward and backward with the residual stream and from an 8-bit
  checkpoint, the checkpoint alone, and the routing of 256 experts with its gradient.

Prints one JSON line per stage with its algorithmic bytes, time and GB/s against the HBM copy
bandwidth in MEASURED_PEAKS.json (or the fallback figure).
"""

from __future__ import annotations

import argparse
import json
import os

import torch

from . import inputs, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def hbm_peak():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        with open(p) as f:
            return float(json.load(f)["hbm_gbs"]), "measured"
    return 6650.0, "fallback"


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--iters", type=int, default=20)
    args = ap.parse_args()
    peak, src = hbm_peak()
    wl = inputs.WORKLOADS["gpt-oss-20b-moe-T8192"]
    inp = inputs.make_workload(wl, 0)
    dev = torch.device("cuda", 0)

    # ---- standalone dequantization of the gate_up weights -------------------------------
    blocks = inp["gu_blocks"].to(dev).reshape(-1, wl.H // 2)
    scales = inp["gu_scales"].to(dev).reshape(-1, wl.H // 32)
    rows, K = blocks.shape[0], wl.H
    out = torch.empty(rows, K, dtype=torch.bfloat16, device=dev)
    for _ in range(3):
        moe.dequantize(blocks, scales, out=out)
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(args.iters):
        moe.dequantize(blocks, scales, out=out)
    e1.record()
    torch.cuda.synchronize()
    ms = e0.elapsed_time(e1) / args.iters
    nbytes = rows * K * (0.5 + 1 / 32 + 2.0)
    print(json.dumps({"stage": "dequant", "rows": rows, "K": K, "bytes": nbytes, "ms": ms,
                      "gbs": nbytes / (ms / 1e3) / 1e9, "frac_of_hbm": nbytes / (ms / 1e3) / 1e9 / peak,
                      "peak_gbs": peak, "peak_source": src}), flush=True)
    del out, blocks, scales
    torch.cuda.empty_cache()

    # ---- gathers and combines of a layer step ------------------------------------------
    shape = moe.MoeShape(wl.T, wl.H, wl.I, wl.E, wl.k)
    w = moe.weights_to(inp, dev)
    wt = moe.transpose_weights(shape, w)
    x, lg, dy = inp["x"].to(dev), inp["logits"].to(dev), inp["dy"].to(dev)
    ws = moe.alloc_workspace(shape, dev)
    y = torch.empty(wl.T, wl.H, dtype=torch.bfloat16, device=dev)
    for _ in range(3):
        moe.forward(shape, w, x, lg, ws, y=y)
        moe.backward_input(shape, w, wt, dy, ws)
    torch.cuda.synchronize()
    moe.profile_begin()
    for _ in range(args.iters):
        moe.forward(shape, w, x, lg, ws, y=y)
        moe.backward_input(shape, w, wt, dy, ws)
    kt = moe.profile_end()
    A, T, H = wl.T * wl.k, wl.T, wl.H
    stages = (("gather_x", A * H * 2.0 * 2),
              ("combine_y", (A + T) * H * 2.0),
              ("gather_dy_dw", A * H * 2.0 * 3 + A * 4.0),
              ("combine_dx", (A + T) * H * 2.0))
    for name, nbytes in stages:
        launches, tot = kt[name]
        ms = tot / launches
        print(json.dumps({"stage": name, "bytes": nbytes, "ms": ms,
                          "gbs": nbytes / (ms / 1e3) / 1e9,
                          "frac_of_hbm": nbytes / (ms / 1e3) / 1e9 / peak,
                          "peak_gbs": peak, "peak_source": src}), flush=True)
    del w, wt, x, lg, dy, ws, y
    torch.cuda.empty_cache()
    edge(args.iters, peak, src)


def edge(iters, peak, src):
    """The operators at the block's edge; inputs of several hundred MB, past L2."""
    T, H, E, k = 32768, 2880, 256, 8
    x, y, d, g = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(4))
    weight = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    f = moe.norm_forward(x, weight, weight, y=y, checkpoint="e4m3")
    cp, dx = f.checkpoint, torch.empty_like(x)
    ws = torch.empty(moe.norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    grads = dict(dx=dx, d_weight=torch.empty(H, device="cuda"), d_bias=torch.empty(H, device="cuda"),
                 ws=ws)
    outs = dict(out=f.out, mean=f.mean, rstd=f.rstd)
    logits = torch.randn(T, E, device="cuda")
    r = moe.Routing(k, "sigmoid", 8, 4, 2)
    idx, w = moe.route(r, logits)
    dl, cells, packed = torch.empty_like(logits), T * H, 1 + 1 / 32
    stages = (
        ("norm_forward", cells * 4.0, lambda: moe.norm_forward(x, weight, weight, **outs)),
        ("norm_forward_residual", cells * 8.0,
         lambda: moe.norm_forward(x, weight, weight, y=y, x_out=f.x_out, **outs)),
        ("norm_forward_residual_checkpoint", cells * (8.0 + packed),
         lambda: moe.norm_forward(x, weight, weight, y=y, x_out=f.x_out, checkpoint=cp, **outs)),
        ("norm_forward_from_checkpoint", cells * (2.0 + packed),
         lambda: moe.norm_forward(cp, weight, weight, **outs)),
        ("norm_backward", cells * 6.0,
         lambda: moe.norm_backward(d, x, f.mean, f.rstd, weight, **grads)),
        ("norm_backward_residual", cells * 8.0,
         lambda: moe.norm_backward(d, x, f.mean, f.rstd, weight, g=g, **grads)),
        ("norm_backward_residual_from_checkpoint", cells * (6.0 + packed),
         lambda: moe.norm_backward(d, cp, f.mean, f.rstd, weight, g=g, **grads)),
        ("checkpoint_pack", cells * (2.0 + packed), lambda: moe.checkpoint_pack(x, out=cp)),
        ("checkpoint_unpack", cells * (2.0 + packed), lambda: moe.checkpoint_unpack(cp, out=dx)),
        ("route", T * (4.0 * E + 8 * k), lambda: moe.route(r, logits, None, idx, w)),
        ("route_backward", T * (4.0 * E + 12 * k),
         lambda: moe.route_backward(r, logits, idx, w, w, dl)),
    )
    for name, nbytes, call in stages:
        for _ in range(3):
            call()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        e0.record()
        for _ in range(iters):
            call()
        e1.record()
        torch.cuda.synchronize()
        ms = e0.elapsed_time(e1) / iters
        gbs = nbytes / (ms / 1e3) / 1e9
        print(json.dumps({"stage": name, "bytes": nbytes, "ms": ms, "gbs": gbs,
                          "frac_of_hbm": gbs / peak, "peak_gbs": peak, "peak_source": src}),
              flush=True)


if __name__ == "__main__":
    main()
