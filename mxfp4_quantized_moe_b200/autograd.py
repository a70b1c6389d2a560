"""The expert block as a torch.autograd.Function, for adapter training over frozen MXFP4 experts.

    layer = MoeLayer(shape, weights)              # packed weights on the GPU, prepared once
    y = moe_block(x, logits, layer)               # x bf16 [T,H], logits fp32 [T,E] (may need grad)
    y.backward(dy)                                # x.grad and logits.grad; no weight gradient

The forward and backward are the library's entry points; this module only wires them into
autograd.  The forward leaves the state the backward needs (routing, permutation, GLU output
and derivative factors) in the layer's workspace, so a layer's backward must follow its own
forward before that layer runs forward again: one MoeLayer per block in the graph, or
recompute the forward before the backward (see stack.py).

Around the block, in the same graph:

    n = norm(x, weight, bias)                     # or (n, x_out) = norm(..., residual=y)
    idx, w = route(logits, routing, bias)         # moe.Routing: scores, groups, balance bias
    y = moe_block_routed(n, idx, w, layer)        # the block on that routing

norm(..., checkpoint="e4m3" | "int8") keeps the rows for the backward in 8 bits, as the stack does.
The backwards of these cannot be captured into a CUDA graph (an eager graph over the same leaves
would end the process); capture moe.norm_backward, moe.route_backward and moe.backward_input
instead.

Source: "Add MXFP4 training support via a dequantize-on-the-fly fallback" (sections "What this
does" and "Relation to the backward triton kernels": gradients reach the inputs through the
expert math; the frozen quantized base gets no weight gradient).
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import moe


class MoeLayer:
    """One block's frozen packed weights with its transposed backward copy and workspace."""

    def __init__(self, shape: moe.MoeShape, weights: dict, device=None):
        self.shape = shape
        self.w = weights
        dev = weights["gu_blocks"].device if device is None else torch.device(device)
        self.wt = moe.transpose_weights(shape, weights)
        self.ws = moe.alloc_workspace(shape, dev)
        self.forwards = 0       # forwards run on this workspace
        self.consumed = True    # the latest forward's state was used by a backward


class _MoeBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x: torch.Tensor, logits: torch.Tensor, layer: MoeLayer):
        y = moe.forward(layer.shape, layer.w, x.contiguous(), logits.contiguous(), layer.ws)
        layer.forwards += 1
        layer.consumed = False
        ctx.layer = layer
        ctx.forward_id = layer.forwards
        return y

    @staticmethod
    def backward(ctx, dy: torch.Tensor):
        layer = ctx.layer
        if layer.forwards != ctx.forward_id or layer.consumed:
            raise RuntimeError("MoeLayer: the workspace no longer holds this forward's state "
                               "(another forward or backward of the layer ran in between)")
        dx, _, d_logits = moe.backward_input(layer.shape, layer.w, layer.wt,
                                             dy.to(torch.bfloat16).contiguous(), layer.ws)
        layer.consumed = True
        return dx, d_logits, None


def moe_block(x: torch.Tensor, logits: torch.Tensor, layer: MoeLayer) -> torch.Tensor:
    """y = MoE(x, logits) with gradients to x and logits (bf16 x, fp32 logits, bf16 y)."""
    return _MoeBlock.apply(x, logits, layer)


def _refuse_capture(what: str, instead: str) -> None:
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what}: the autograd backward cannot be captured into a CUDA graph; "
                           f"capture {instead}")


class _MoeBlockRouted(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_idx, topk_w, layer: MoeLayer):
        y = moe.forward_routed(layer.shape, layer.w, x.contiguous(), topk_idx.contiguous(),
                               topk_w.contiguous(), layer.ws)
        layer.forwards += 1
        layer.consumed = False
        ctx.layer = layer
        ctx.forward_id = layer.forwards
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        layer = ctx.layer
        _refuse_capture("moe_block_routed", "moe.backward_input")
        if layer.forwards != ctx.forward_id or layer.consumed:
            raise RuntimeError("MoeLayer: the workspace no longer holds this forward's state "
                               "(another forward or backward of the layer ran in between)")
        dx, d_topk_w, _ = moe.backward_input(layer.shape, layer.w, layer.wt,
                                             dy.to(torch.bfloat16).contiguous(), layer.ws,
                                             want_d_logits=False)
        layer.consumed = True
        return dx, None, d_topk_w, None


def moe_block_routed(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                     layer: MoeLayer) -> torch.Tensor:
    """The block on a given routing (topk_idx int32 [T, k], topk_w fp32 [T, k]), with gradients to
    x and topk_w."""
    return _MoeBlockRouted.apply(x, topk_idx, topk_w, layer)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, routing, bias):
        logits = logits.contiguous()
        idx, w = moe.route(routing, logits, bias)
        ctx.mark_non_differentiable(idx)
        ctx.save_for_backward(logits, idx, w)
        ctx.routing = routing
        return idx, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, d_w):
        _refuse_capture("route", "moe.route_backward")
        logits, idx, w = ctx.saved_tensors
        return moe.route_backward(ctx.routing, logits, idx, w, d_w.contiguous()), None, None


def route(logits: torch.Tensor, routing: moe.Routing, bias: torch.Tensor | None = None):
    """moe.route with the weights' gradient to the logits: (topk_idx, topk_w) of fp32 logits
    [T, E].  The selection and the bias carry no gradient."""
    return _Route.apply(logits, routing, None if bias is None else bias.detach())


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, kind, eps, checkpoint):
        rows = x.contiguous().view(-1, x.shape[-1])
        y = None if residual is None else residual.contiguous().view(rows.shape)
        w = None if weight is None else weight.contiguous()
        f = moe.norm_forward(rows, w, None if bias is None else bias.contiguous(), kind=kind,
                             eps=eps, y=y, checkpoint=checkpoint)
        # fresh tensors in x's shape, no views of them: a view that a Function returns may not be
        # changed in place
        out = f.out.resize_(x.shape)
        x_out = None if y is None else f.x_out.resize_(x.shape)
        if checkpoint:
            ctx.save_for_backward(f.checkpoint.codes, f.checkpoint.scales, w)
        else:
            ctx.save_for_backward(rows if y is None else x_out, w, f.mean, f.rstd)
        ctx.kind, ctx.eps, ctx.checkpoint, ctx.shape = kind, eps, checkpoint, x.shape
        ctx.bias_type = None if bias is None else bias.dtype
        return out if residual is None else (out, x_out)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_x_out=None):
        _refuse_capture("norm", "moe.norm_backward")
        if ctx.checkpoint:
            # the gradient at the rows that are kept: x_hat has mean 0 and variance 1 only with
            # their own statistics
            kept, scales, w = ctx.saved_tensors
            rows = moe.Checkpoint(kept, scales, ctx.checkpoint)
            f = moe.norm_forward(rows, kind=ctx.kind, eps=ctx.eps, dtype=d_out.dtype)
            mean, rstd = f.mean, f.rstd
        else:
            kept, w, mean, rstd = ctx.saved_tensors
            rows = kept = kept.view(-1, kept.shape[-1])
        shape = kept.shape
        g = None if d_x_out is None else d_x_out.contiguous().view(shape)
        params = (w is not None and ctx.needs_input_grad[1]) or ctx.needs_input_grad[2]
        dx, d_weight, d_bias = moe.norm_backward(
            d_out.contiguous().view(shape), rows, mean, rstd, w, kind=ctx.kind, g=g, params=params,
            d_bias=(torch.empty(shape[1], dtype=torch.float32, device=kept.device)
                    if params and ctx.kind == "rms" and ctx.needs_input_grad[2] else None))
        dx = dx.view(ctx.shape)
        return (dx if ctx.needs_input_grad[0] else None,
                d_weight.to(w.dtype) if params and ctx.needs_input_grad[1] else None,
                d_bias.to(ctx.bias_type) if params and ctx.needs_input_grad[2] else None,
                dx if ctx.needs_input_grad[3] else None, None, None, None)


def norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
         residual: torch.Tensor | None = None, kind: str = "layer", eps: float = 1e-5,
         checkpoint: str | None = None):
    """Layer or rms norm over the last dimension of x (bf16 or fp32), with gradients to x, weight,
    bias and residual.  With a residual: (norm(x + residual), x + residual).  checkpoint ("e4m3" or
    "int8", the last dimension a multiple of 32): the rows are kept in 8 bits, and the backward is
    the norm's gradient at the rows that these stand for (one more pass over them, for their
    statistics)."""
    return _Norm.apply(x, weight, bias, residual, kind, eps, checkpoint)
