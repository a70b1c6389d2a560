"""A residual stack of MXFP4 MoE blocks with a recompute-per-block backward.

    x_{l+1} = x_l + MoE_l(x_l, logits_l),   logits_l = x_l W_r^l + b_r^l   (fp32)

The blocks are the library's entry points (mxfp4_moe_forward / mxfp4_moe_backward_input);
the caller's side of the block boundary is two more of its kernels: mxfp4_moe_residual_router
forms x_{l+1} = bf16(x_l + y_l) and the next block's logits from one read of x_l and y_l, and
mxfp4_moe_grad_chain forms g_l below.  The backward is activation checkpointing at block
granularity: the forward keeps only each block's input x_l (bf16); the backward re-runs
block l's forward from x_l to refill the one shared workspace, then runs its input-gradient
backward, so at most one block's transients are alive at any time.

Chain rule per block (g_{l+1} = dL/dx_{l+1}):
    g_l = g_{l+1} + dX_moe_l + d_logits_l (W_r^l)^T
with dX_moe_l and d_logits_l returned by the block's backward for upstream gradient g_{l+1}.
Sums are taken in fp32 and rounded to bf16 once per block, like the residual stream.

Options put the rest of a decoder layer's MoE half around the blocks:

    norm        n_l = norm(x_l; weight_l, bias_l) is what the block and its router take; the
                residual add, the next norm and the checkpoint are one kernel, and the backward
                also returns the norms' gradients (`norm_grads`);
    routing     the experts are chosen by a `moe.Routing` (scores, groups, the block's
                route_bias) instead of the softmax over the k largest logits;
    checkpoint  "e4m3" or "int8": x_l is kept in 8 bits between the forward and the backward;
                the recompute and the norm's backward read it as it is stored.

The forward checkpoints each block's input x_l together with its logits_l (T x E fp32, a
few MB a block), so the recompute needs no router call.  The block functions and the two
caller-side steps are injectable, so that the chaining itself can be checked on the CPU
against an fp64 reference without a GPU.

Source: "Add MXFP4 training support via a dequantize-on-the-fly fallback" (the MoE block of
a decoder layer trained with gradient checkpointing over packed frozen weights).
"""

from __future__ import annotations

import argparse
import json
from dataclasses import dataclass
from typing import Callable

import torch


@dataclass
class StackBlock:
    """One block's operands on the device: packed weights (dict as `moe.weights_to` returns),
    the transposed copy for the backward, the router linear W_r [H,E], b_r [E], and, for the
    stack's options, the norm's weight and bias [H] and the routing's balance bias fp32 [E]."""
    w: dict
    wt: torch.Tensor | None
    w_r: torch.Tensor
    b_r: torch.Tensor
    norm_w: torch.Tensor | None = None
    norm_b: torch.Tensor | None = None
    route_bias: torch.Tensor | None = None


class MoeStack:
    """Forward and recompute-per-block backward over a list of blocks.

    `norm` ("layer" or "rms", with `eps`), `routing` (a `moe.Routing`) and `checkpoint` ("e4m3" or
    "int8") are the options above.

    `block_forward(l, x, how) -> y` and `block_backward(l, g) -> (dx, d_logits)` default to
    the library's entry points on one shared workspace; `how` is the block's logits, or with a
    routing the pair (topk_idx, topk_w), and the backward then returns (dx, None, d_topk_w).
    `block_backward` sees the workspace that the immediately preceding `block_forward(l, ...)`
    left.
    `residual_router(x, y, w_r, b_r) -> (x + y or None, logits or None)` (y None: logits of
    x; w_r None: no logits) and `grad_chain(g, dx, d_logits, w_r)` default to the library's
    mxfp4_moe_residual_router and mxfp4_moe_grad_chain; `ops` holds the options' functions
    (norm_forward, norm_backward, route, route_backward, checkpoint_pack, checkpoint_unpack) and
    defaults to the `moe` module."""

    def __init__(self, shape, blocks: list[StackBlock], device=None,
                 block_forward: Callable | None = None, block_backward: Callable | None = None,
                 residual_router: Callable | None = None, grad_chain: Callable | None = None,
                 norm: str | None = None, eps: float = 1e-5, routing=None,
                 checkpoint: str | None = None, ops=None):
        self.shape = shape
        self.blocks = blocks
        self.norm, self.eps, self.routing, self.checkpoint = norm, eps, routing, checkpoint
        self.norm_grads: list = []
        if routing is not None and shape is not None and routing.k != shape.k:
            raise ValueError("the routing's k is not the blocks'")
        if ops is None and (norm or routing or checkpoint):
            from . import moe as ops
        self.ops = ops
        if residual_router is None or grad_chain is None:
            from . import moe
            self._moe = moe
        self.residual_router = residual_router or self._lib_residual_router
        self.grad_chain = grad_chain or self._lib_grad_chain
        if block_forward is None or block_backward is None:
            from . import moe
            self._moe = moe
            dev = blocks[0].w_r.device if device is None else torch.device(device)
            self.ws = moe.alloc_workspace(shape, dev)
            T, H = shape.T, shape.H
            self._y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
            self._dx = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
            self._dtw = torch.empty(T, shape.k, dtype=torch.float32, device=dev)
            self._dl = torch.empty(T, shape.E, dtype=torch.float32, device=dev)
        self.block_forward = block_forward or self._lib_forward
        self.block_backward = block_backward or self._lib_backward

    # ---- the library's entry points ------------------------------------------------------
    def _lib_forward(self, l, x, how):
        if self.routing is not None:
            return self._moe.forward_routed(self.shape, self.blocks[l].w, x, *how, self.ws,
                                            y=self._y)
        return self._moe.forward(self.shape, self.blocks[l].w, x, how, self.ws, y=self._y)

    def _lib_backward(self, l, g):
        b, own = self.blocks[l], self.routing is None
        dx, dtw, dl = self._moe.backward_input(self.shape, b.w, b.wt, g, self.ws, dx=self._dx,
                                               d_topk_w=self._dtw,
                                               d_logits=self._dl if own else None,
                                               want_d_logits=own)
        return dx, dl, dtw

    def _lib_residual_router(self, x, y, w_r, b_r):
        return self._moe.residual_router(x, y, w_r, b_r)

    def _lib_grad_chain(self, g, dx, d_logits, w_r):
        return self._moe.grad_chain(g, dx, d_logits, w_r)

    # ---- the stack -----------------------------------------------------------------------
    def _enter(self, l, x, y):
        """Block l's input from the previous one's input and output (y None: x itself): the
        residual stream, what the block takes, its logits, and what is kept of the stream."""
        b = self.blocks[l]
        if self.norm:
            f = self.ops.norm_forward(x, b.norm_w, b.norm_b, kind=self.norm, eps=self.eps, y=y,
                                      checkpoint=self.checkpoint)
            x = x if y is None else f.x_out
            logits = self.residual_router(f.out, None, b.w_r, b.b_r)[1]
            return x, f.out, logits, f.checkpoint if self.checkpoint else x
        x_next, logits = self.residual_router(x, y, b.w_r, b.b_r)
        x = x if y is None else x_next
        return x, x, logits, self.ops.checkpoint_pack(x, self.checkpoint) if self.checkpoint else x

    def _choose(self, l, logits):
        if self.routing is None:
            return logits
        return self.ops.route(self.routing, logits, self.blocks[l].route_bias)

    def forward(self, x: torch.Tensor, tap: Callable | None = None):
        """Returns (x_L, saved); saved[l] begins with (x_l or its checkpoint, logits_l) for the
        recompute and goes on with the routing, where the stack has one.  `tap(l, dict)` sees
        each block's x (what the block takes), logits, y."""
        saved = []
        y = None
        for l in range(len(self.blocks)):
            x, n, logits, kept = self._enter(l, x, y)
            how = self._choose(l, logits)
            saved.append((kept, logits) if self.routing is None else (kept, logits, *how))
            y = self.block_forward(l, n, how)
            if tap is not None:
                tap(l, {"x": n, "logits": logits, "y": y, "rows": x, "how": how})
        return self.residual_router(x, y, None, None)[0], saved

    def backward(self, dy: torch.Tensor, saved: list, tap: Callable | None = None):
        """dL/dx_0 from dL/dx_L, re-running each block's forward from its saved input.  With a
        norm, norm_grads[l] receives (d_weight, d_bias) of block l's."""
        g = dy
        self.norm_grads = [None] * len(self.blocks)
        for l in reversed(range(len(self.blocks))):
            b = self.blocks[l]
            kept, logits, *how = saved[l]
            if self.norm:
                f = self.ops.norm_forward(kept, b.norm_w, b.norm_b, kind=self.norm, eps=self.eps,
                                          **({"dtype": dy.dtype} if self.checkpoint else {}))
                n = f.out
            else:
                n = self.ops.checkpoint_unpack(kept, dy.dtype) if self.checkpoint else kept
            # recompute: refills the block's saved state
            self.block_forward(l, n, tuple(how) if how else logits)
            out = self.block_backward(l, g)
            dx_moe, d_logits = out[0], out[1]
            if self.routing is not None:
                d_logits = self.ops.route_backward(self.routing, logits, *how, out[2])
            if tap is not None:
                tap(l, {"g": g, "dx": dx_moe, "d_logits": d_logits,
                        "d_w": out[2] if len(out) > 2 else None, "x": n})
            if self.norm:
                dn = self.grad_chain(dx_moe, None, d_logits, b.w_r)
                g, self.norm_grads[l] = self._norm_backward(dn, kept, f, b, g)
            else:
                g = self.grad_chain(g, dx_moe, d_logits, b.w_r)
        return g

    def _norm_backward(self, dn, kept, f, b, g):
        dx, d_weight, d_bias = self.ops.norm_backward(dn, kept, f.mean, f.rstd, b.norm_w,
                                                      kind=self.norm, g=g)
        return dx, (d_weight, d_bias)


def build_stack(wl, seed: int = 0, device="cuda", layers: int | None = None,
                norm: str | None = None, routing=None):
    """Device blocks of a stacked workload (layer l drawn from seed + l), the stack input x
    (layer 0's x draw) and the upstream gradient dY (layer 0's dY draw).  With a norm or a routing,
    the norms' parameters (near 1 and 0) and the balance biases (near 0) are drawn as well."""
    from . import inputs, moe
    n_layers = wl.layers if layers is None else layers
    shape = moe.MoeShape(wl.T, wl.H, wl.I, wl.E, wl.k)
    blocks, x, dy = [], None, None
    for l in range(n_layers):
        inp = inputs.make_workload(wl, seed, layer=l, with_dy=(l == 0))
        if l == 0:
            x, dy = inp["x"].to(device), inp["dy"].to(device)
        w = moe.weights_to(inp, device)
        wt = moe.transpose_weights(shape, w)
        b = StackBlock(w, wt, inp["w_r"].to(device), inp["b_r"].to(device))
        gen = torch.Generator().manual_seed(seed + l)
        if norm:
            b.norm_w = (1.0 + 0.1 * torch.randn(wl.H, generator=gen)).to(torch.bfloat16).to(device)
            if norm == "layer":
                b.norm_b = (0.1 * torch.randn(wl.H, generator=gen)).to(torch.bfloat16).to(device)
        if routing is not None:
            b.route_bias = (0.01 * torch.randn(wl.E, generator=gen)).to(device)
        blocks.append(b)
        del inp
    return shape, blocks, x, dy


def main():
    """Times the stack's forward + recompute backward on one GPU and reports peak memory."""
    from . import inputs
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="gpt-oss-20b-moe-stack24-T32768")
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--warmup", type=int, default=1)
    ap.add_argument("--norm", choices=("layer", "rms"), help="a norm in front of every block")
    ap.add_argument("--scores", choices=("softmax", "sigmoid"),
                    help="routing with these scores and a balance bias")
    ap.add_argument("--checkpoint", choices=("e4m3", "int8"),
                    help="block inputs kept in 8 bits between forward and backward")
    args = ap.parse_args()
    wl = inputs.WORKLOADS[args.workload]
    routing = None
    if args.scores:
        from . import moe
        routing = moe.Routing(wl.k, args.scores)
    shape, blocks, x, dy = build_stack(wl, norm=args.norm, routing=routing)
    st = MoeStack(shape, blocks, norm=args.norm, routing=routing, checkpoint=args.checkpoint)
    for _ in range(args.warmup):
        out, saved = st.forward(x)
        st.backward(dy, saved)
        del out, saved
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(args.steps):
        out, saved = st.forward(x)
        st.backward(dy, saved)
        del out, saved
    e1.record()
    torch.cuda.synchronize()
    ms = e0.elapsed_time(e1) / args.steps
    A = wl.T * wl.k
    model_flop = 12.0 * A * wl.H * wl.I * wl.layers
    exec_flop = model_flop * 1.5  # the recompute repeats every block's forward (half the work)
    print(json.dumps({
        "workload": wl.name, "layers": wl.layers, "norm": args.norm, "scores": args.scores,
        "checkpoint": args.checkpoint, "ms_per_step": ms,
        "tokens_per_s": wl.T / (ms / 1e3),
        "model_tflops": model_flop / (ms / 1e3) / 1e12,
        "executed_tflops": exec_flop / (ms / 1e3) / 1e12,
        "peak_memory_gb": torch.cuda.max_memory_allocated() / 1e9,
        "resident_weights_gb": sum(
            sum(int(t.numel()) * t.element_size() for t in b.w.values()) +
            int(b.wt.numel()) * b.wt.element_size() for b in blocks) / 1e9,
    }), flush=True)


if __name__ == "__main__":
    main()
