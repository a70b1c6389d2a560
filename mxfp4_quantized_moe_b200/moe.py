"""Torch-facing wrappers over the C ABI (device memory and streams come from torch).

Each function checks shapes and dtypes, hands raw device pointers and the current CUDA
stream to the library, and returns torch tensors.  All computation happens in the
library's kernels.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
from dataclasses import dataclass
from functools import lru_cache
from typing import NamedTuple

import torch

from . import _lib, build
from ._lib import Dims, Weights, check, lib


def _load_edge():
    """The binding module of this torch and Python (csrc/binding.cpp); like the library, it fails
    loudly where it is missing."""
    if not os.path.exists(build.BINDING):
        raise ImportError(
            f"{build.BINDING} is missing: build it with `python -m mxfp4_quantized_moe_b200.build` "
            "(there is no fallback implementation)")
    spec = importlib.util.spec_from_file_location(f"{__package__}._edge", build.BINDING)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_edge = _load_edge()
_edge.bind(*(ctypes.cast(getattr(lib, "mxfp4_moe_" + name), ctypes.c_void_p).value for name in (
    "route", "route_backward", "norm_forward", "norm_workspace_size", "norm_backward",
    "checkpoint_pack", "checkpoint_unpack")))


@dataclass
class MoeShape:
    T: int
    H: int
    I: int
    E: int
    k: int
    glu_alpha: float = 1.702
    glu_limit: float = 7.0
    # forward gate_up operands: 0 = bf16 (weights dequantized on the fly), 1 = block-scaled
    # (E2M1 weights as stored against E4M3 hi / lo token parts with UE8M0 block scales)
    gate_up_format: int = 0

    def dims(self) -> Dims:
        return Dims(self.T, self.H, self.I, self.E, self.k, self.glu_alpha, self.glu_limit,
                    self.gate_up_format)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _weights(w: dict) -> Weights:
    for key, dt in (("gu_blocks", torch.uint8), ("gu_scales", torch.uint8),
                    ("gu_bias", torch.bfloat16), ("dn_blocks", torch.uint8),
                    ("dn_scales", torch.uint8), ("dn_bias", torch.bfloat16)):
        if w[key].dtype != dt:
            raise TypeError(f"{key} must be {dt}")
    return Weights(_ptr(w["gu_blocks"]), _ptr(w["gu_scales"]), _ptr(w["gu_bias"]),
                   _ptr(w["dn_blocks"]), _ptr(w["dn_scales"]), _ptr(w["dn_bias"]))


def workspace_bytes(shape: MoeShape) -> int:
    n = ctypes.c_size_t()
    check(lib.mxfp4_moe_workspace_size(ctypes.byref(shape.dims()), ctypes.byref(n)),
          "mxfp4_moe_workspace_size")
    return n.value


def transposed_weights_bytes(shape: MoeShape) -> int:
    n = ctypes.c_size_t()
    check(lib.mxfp4_moe_transposed_weights_size(ctypes.byref(shape.dims()), ctypes.byref(n)),
          "mxfp4_moe_transposed_weights_size")
    return n.value


def alloc_workspace(shape: MoeShape, device="cuda") -> torch.Tensor:
    return torch.zeros(workspace_bytes(shape), dtype=torch.uint8, device=device)


def transpose_weights(shape: MoeShape, w: dict, out: torch.Tensor | None = None, stream=None):
    n = transposed_weights_bytes(shape)
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w["gu_blocks"].device)
    check(lib.mxfp4_moe_transpose_weights(ctypes.byref(shape.dims()), ctypes.byref(_weights(w)),
                                          _ptr(out), out.numel(), _stream(stream)),
          "mxfp4_moe_transpose_weights")
    return out


def forward(shape: MoeShape, w: dict, x: torch.Tensor, logits: torch.Tensor, ws: torch.Tensor,
            y: torch.Tensor | None = None, topk_idx: torch.Tensor | None = None,
            topk_w: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    T, H = shape.T, shape.H
    if x.shape != (T, H) or x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 [T, H]")
    if logits.shape != (T, shape.E) or logits.dtype != torch.float32:
        raise ValueError("logits must be fp32 [T, E]")
    if y is None:
        y = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    check(lib.mxfp4_moe_forward(ctypes.byref(shape.dims()), ctypes.byref(_weights(w)), _ptr(x),
                                _ptr(logits), _ptr(y), _ptr(topk_idx), _ptr(topk_w), _ptr(ws),
                                ws.numel(), _stream(stream)), "mxfp4_moe_forward")
    return y


def backward_input(shape: MoeShape, w: dict, wt: torch.Tensor, dy: torch.Tensor,
                   ws: torch.Tensor, dx: torch.Tensor | None = None,
                   d_topk_w: torch.Tensor | None = None, d_logits: torch.Tensor | None = None,
                   want_d_logits: bool = True, stream=None):
    T, H = shape.T, shape.H
    if dy.shape != (T, H) or dy.dtype != torch.bfloat16:
        raise ValueError("dy must be bf16 [T, H]")
    dev = dy.device
    if dx is None:
        dx = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if d_topk_w is None:
        d_topk_w = torch.empty(T, shape.k, dtype=torch.float32, device=dev)
    if d_logits is None and want_d_logits:
        d_logits = torch.empty(T, shape.E, dtype=torch.float32, device=dev)
    check(lib.mxfp4_moe_backward_input(ctypes.byref(shape.dims()), ctypes.byref(_weights(w)),
                                       _ptr(wt), wt.numel(), _ptr(dy), _ptr(ws), ws.numel(),
                                       _ptr(dx), _ptr(d_topk_w), _ptr(d_logits),
                                       _stream(stream)), "mxfp4_moe_backward_input")
    return dx, d_topk_w, d_logits


def dequantize(blocks: torch.Tensor, scales: torch.Tensor, stream=None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [rows, K] from packed uint8 [rows, K/2] and UE8M0 scales [rows, K/32]."""
    rows = blocks.numel() // blocks.shape[-1]
    K = blocks.shape[-1] * 2
    if scales.numel() != rows * (K // 32):
        raise ValueError("scales do not match blocks")
    if out is None:
        out = torch.empty(*blocks.shape[:-1], K, dtype=torch.bfloat16, device=blocks.device)
    elif out.numel() != rows * K or out.dtype != torch.bfloat16:
        raise ValueError("out must be bf16 with rows * K elements")
    check(lib.mxfp4_moe_dequantize(_ptr(blocks), _ptr(scales), rows, K, _ptr(out),
                                   _stream(stream)), "mxfp4_moe_dequantize")
    return out


def grouped_matmul(off: torch.Tensor, x: torch.Tensor, blocks: torch.Tensor,
                   scales: torch.Tensor, N: int, transposed: bool = False,
                   err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[r] = x[r] W_e^T for the rows r of expert e (off: int32 [E+1] on the device)."""
    E = off.numel() - 1
    A, K = x.shape
    if x.dtype != torch.bfloat16 or off.dtype != torch.int32:
        raise TypeError("x must be bf16 and off int32")
    out = torch.empty(A, N, dtype=torch.bfloat16, device=x.device)
    check(lib.mxfp4_moe_grouped_matmul(E, N, K, A, _ptr(off), _ptr(x), _ptr(blocks),
                                       _ptr(scales), 1 if transposed else 0, _ptr(out),
                                       _ptr(err), _stream(stream)), "mxfp4_moe_grouped_matmul")
    return out


def device_check(ws: torch.Tensor, stream=None) -> tuple[int, int]:
    """Synchronize and read (then clear) the device error word: (code, where)."""
    where = ctypes.c_int32(0)
    rc = lib.mxfp4_moe_check(_ptr(ws), _stream(stream), ctypes.byref(where))
    return rc, where.value


def interleave_gate_up(shape: MoeShape, blocks: torch.Tensor, scales: torch.Tensor,
                       bias: torch.Tensor, stream=None):
    """Stacked gate_up (rows [gates; ups]) -> interleaved (gate j at 2j, up j at 2j+1);
    returns new (blocks, scales, bias) tensors."""
    ob, os_, obias = torch.empty_like(blocks), torch.empty_like(scales), torch.empty_like(bias)
    check(lib.mxfp4_moe_interleave_gate_up(ctypes.byref(shape.dims()), _ptr(blocks), _ptr(scales),
                                           _ptr(bias), _ptr(ob), _ptr(os_), _ptr(obias),
                                           _stream(stream)), "mxfp4_moe_interleave_gate_up")
    return ob, os_, obias


def residual_router(x: torch.Tensor, y: torch.Tensor | None, w_r: torch.Tensor | None,
                    b_r: torch.Tensor | None = None, x_out: torch.Tensor | None = None,
                    logits: torch.Tensor | None = None, stream=None):
    """The residual stream between stacked blocks in one kernel: x_out = bf16(x + y) when y is
    given, and logits = (x_out or x) W_r + b_r in fp32 when w_r is given.  Returns
    (x_out or None, logits or None)."""
    T, H = x.shape
    if x.dtype != torch.bfloat16 or (y is not None and (y.shape != x.shape or y.dtype != x.dtype)):
        raise ValueError("x and y must be bf16 [T, H]")
    E = w_r.shape[1] if w_r is not None else 1
    if w_r is not None:
        if w_r.shape != (H, E) or w_r.dtype != torch.bfloat16:
            raise ValueError("w_r must be bf16 [H, E]")
        if b_r is not None and (b_r.shape != (E,) or b_r.dtype != torch.bfloat16):
            raise ValueError("b_r must be bf16 [E]")
        if logits is None:
            logits = torch.empty(T, E, dtype=torch.float32, device=x.device)
    else:
        logits = None
    if y is not None and x_out is None:
        x_out = torch.empty_like(x)
    if y is None:
        x_out = None
    check(lib.mxfp4_moe_residual_router(T, H, E, _ptr(x), _ptr(y), _ptr(w_r), _ptr(b_r),
                                        _ptr(x_out), _ptr(logits), _stream(stream)),
          "mxfp4_moe_residual_router")
    return x_out, logits


def grad_chain(g: torch.Tensor, dx: torch.Tensor | None, d_logits: torch.Tensor, w_r: torch.Tensor,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16(g + dx + d_logits W_r^T) in fp32, one kernel (out may be g itself; dx None: without
    that term)."""
    T, H = g.shape
    E = w_r.shape[1]
    if g.dtype != torch.bfloat16 or (dx is not None and (dx.shape != g.shape
                                                         or dx.dtype != g.dtype)):
        raise ValueError("g and dx must be bf16 [T, H]")
    if d_logits.shape != (T, E) or d_logits.dtype != torch.float32:
        raise ValueError("d_logits must be fp32 [T, E]")
    if w_r.shape != (H, E) or w_r.dtype != torch.bfloat16:
        raise ValueError("w_r must be bf16 [H, E]")
    if out is None:
        out = torch.empty_like(g)
    check(lib.mxfp4_moe_grad_chain(T, H, E, _ptr(g), _ptr(dx), _ptr(d_logits), _ptr(w_r),
                                   _ptr(out), _stream(stream)), "mxfp4_moe_grad_chain")
    return out


# ---- the operators at the block's edge: routing, the norm, 8-bit checkpoints ----------------
# These run on the device of their tensors (all on one), whichever device is current, on that
# device's current stream or on `stream`; what they allocate belongs to that stream.  Rows and
# vectors are dense; every output that a caller may pass is also what the call returns.  The plain
# call (outputs not given, the present stream and device) goes through _edge in one step; it
# returns None for any other and for every error, and the long way below names it.
_EMPTY = 256  # stands for the null pointer of a tensor without elements; never dereferenced
_F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8,)
_ROWS = (torch.bfloat16, torch.float32)


def _elsewhere(t: torch.Tensor, stream):
    """The context in which a call on t's device allocates and launches; None: the present one."""
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    if stream is None:
        here = t.get_device() == torch._C._cuda_getDevice()
        return None if here else torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError("stream and tensors are on different devices")
    return torch.cuda.stream(stream)


def _current(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)  # current_stream() costs 2 us more


def _tensor(t: torch.Tensor, name: str, shape, dtypes, index: int) -> int:
    """The data pointer of a dense tensor of that shape and type on CUDA device `index`."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    if t.get_device() != index:  # -1 on the host
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    p = t.data_ptr()
    if not p and t.numel():
        raise ValueError(f"{name} has no memory")
    return p or _EMPTY


def _int32(**sizes: int) -> None:
    """The library counts in 32 bits, and ctypes drops what does not fit."""
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name} = {v} does not fit 32 bits")


def _aligned(t: torch.Tensor | None):
    """An input beside a checkpoint, which the kernels read in 16-byte vectors: t, or its copy where
    t begins off such an address (a slice of a larger buffer)."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.detach().clone()


@dataclass
class Routing:
    """How tokens choose their experts (mxfp4_moe_routing in include/mxfp4_moe.h)."""
    k: int
    scores: str = "softmax"    # or "sigmoid"
    groups: int = 1            # experts in equal groups, of which the best `top_groups` stay
    top_groups: int = 1
    group_best: int = 1        # 1 or 2: the largest keys that sum to a group's score
    renormalize: bool = True   # weights divided by the selected scores' sum
    scale: float = 1.0

    def dims(self, T: int, E: int) -> _lib.Routing:
        return _routing_dims(T, E, self.k, self.scores, self.groups, self.top_groups,
                             self.group_best, self.renormalize, self.scale)


@lru_cache(maxsize=1024)  # the library only reads them
def _routing_dims(T, E, k, scores, groups, top_groups, group_best, renormalize, scale):
    if scores not in _lib.SCORES:
        raise ValueError(f"scores must be one of {sorted(_lib.SCORES)}")
    _int32(T=T, E=E, k=k, groups=groups, top_groups=top_groups, group_best=group_best)
    return _lib.Routing(T, E, k, _lib.SCORES[scores], groups, top_groups, group_best,
                        int(renormalize), scale)


def _logits_shape(logits: torch.Tensor):
    if logits.dim() != 2:
        raise ValueError("logits must be fp32 [T, E]")
    T, E = logits.shape
    if T >= 2 ** 31 or E >= 2 ** 31:
        _int32(T=T, E=E)
    return T, E


def route(routing: Routing, logits: torch.Tensor, bias: torch.Tensor | None = None,
          topk_idx: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
          counts: torch.Tensor | None = None, stream=None):
    """(topk_idx int32 [T, k], topk_w fp32 [T, k]) of fp32 logits [T, E] and, where given, a
    balance bias fp32 [E] on the selection.  `counts` (int32 [E]) receives the slots of each
    expert.  Logits or biases of NaN, -inf or the lowest finite value mask an expert: it is
    selected last, with weight 0."""
    if stream is None and topk_idx is None and topk_w is None and counts is None:
        done = _edge.route(routing.k, routing.scores, routing.groups, routing.top_groups,
                           routing.group_best, routing.renormalize, routing.scale, logits, bias)
        if done is not None:
            return done
    T, E = _logits_shape(logits)
    where = _elsewhere(logits, stream)
    if where is not None:
        with where:
            return route(routing, logits, bias, topk_idx, topk_w, counts)
    dev = logits.get_device()
    lp = _tensor(logits, "logits", (T, E), _F32, dev)
    bp = None if bias is None else _tensor(bias, "bias", (E,), _F32, dev)
    cp = None if counts is None else _tensor(counts, "counts", (E,), _I32, dev)
    dims, slots = routing.dims(T, E), (T, routing.k)
    if topk_idx is None:
        topk_idx = logits.new_empty(slots, dtype=torch.int32)
        ip = topk_idx.data_ptr() or _EMPTY
    else:
        ip = _tensor(topk_idx, "topk_idx", slots, _I32, dev)
    if topk_w is None:
        topk_w = logits.new_empty(slots)
        wp = topk_w.data_ptr() or _EMPTY
    else:
        wp = _tensor(topk_w, "topk_w", slots, _F32, dev)
    check(lib.mxfp4_moe_route(dims, lp, bp, ip, wp, cp, _current(dev)), "mxfp4_moe_route")
    return topk_idx, topk_w


def route_backward(routing: Routing, logits: torch.Tensor, topk_idx: torch.Tensor,
                   topk_w: torch.Tensor, d_topk_w: torch.Tensor,
                   d_logits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """d_logits fp32 [T, E] from d_topk_w fp32 [T, k], for what `route` returned on `logits`."""
    if stream is None and d_logits is None:
        done = _edge.route_backward(routing.k, routing.scores, routing.groups, routing.top_groups,
                                    routing.group_best, routing.renormalize, routing.scale, logits,
                                    topk_idx, topk_w, d_topk_w)
        if done is not None:
            return done
    T, E = _logits_shape(logits)
    where = _elsewhere(logits, stream)
    if where is not None:
        with where:
            return route_backward(routing, logits, topk_idx, topk_w, d_topk_w, d_logits)
    slots = (T, routing.k)
    dev = logits.get_device()
    lp = _tensor(logits, "logits", (T, E), _F32, dev)
    ip = _tensor(topk_idx, "topk_idx", slots, _I32, dev)
    wp = _tensor(topk_w, "topk_w", slots, _F32, dev)
    dp = _tensor(d_topk_w, "d_topk_w", slots, _F32, dev)
    if d_logits is None:
        d_logits = torch.empty_like(logits)
        op = d_logits.data_ptr() or _EMPTY
    else:
        op = _tensor(d_logits, "d_logits", (T, E), _F32, dev)
    check(lib.mxfp4_moe_route_backward(routing.dims(T, E), lp, ip, wp, dp, op, _current(dev)),
          "mxfp4_moe_route_backward")
    return d_logits


def forward_routed(shape: MoeShape, w: dict, x: torch.Tensor, topk_idx: torch.Tensor,
                   topk_w: torch.Tensor, ws: torch.Tensor, y: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The block's forward on a given routing in place of its own (topk_idx int32 and topk_w fp32
    [T, k]).  `backward_input(..., want_d_logits=False)` follows it; its d_topk_w goes on to
    `route_backward`."""
    where = _elsewhere(x, stream)
    if where is not None:
        with where:
            return forward_routed(shape, w, x, topk_idx, topk_w, ws, y)
    dev = x.get_device()
    rows, slots = (shape.T, shape.H), (shape.T, shape.k)
    xp = _tensor(x, "x", rows, (torch.bfloat16,), dev)
    ip = _tensor(topk_idx, "topk_idx", slots, _I32, dev)
    wp = _tensor(topk_w, "topk_w", slots, _F32, dev)
    if ws.get_device() != dev or any(t.get_device() != dev for t in w.values()):
        raise ValueError(f"ws and the weights must be on cuda:{dev}")
    if y is None:
        y = torch.empty_like(x)
    check(lib.mxfp4_moe_forward_routed(
        shape.dims(), _weights(w), xp, ip, wp, _tensor(y, "y", rows, (torch.bfloat16,), dev),
        _ptr(ws), ws.numel() * ws.element_size(), _current(dev)), "mxfp4_moe_forward_routed")
    return y


@dataclass
class Checkpoint:
    """Rows in 8 bits: codes uint8 [T, H] and a UE8M0 scale uint8 [T, H/32] per 32 features;
    format "e4m3" (MXFP8) or "int8" (MXINT8)."""
    codes: torch.Tensor
    scales: torch.Tensor
    format: str = "e4m3"

    @staticmethod
    def empty(T: int, H: int, format: str = "e4m3", device="cuda") -> "Checkpoint":
        if H % 32:
            raise ValueError("a checkpoint needs H to be a multiple of 32")
        return Checkpoint(torch.empty((T, H), dtype=torch.uint8, device=device),
                          torch.empty((T, H // 32), dtype=torch.uint8, device=device), format)

    @staticmethod
    def _beside(x: torch.Tensor, format: str) -> "Checkpoint":
        T, H = x.shape
        if H % 32:
            raise ValueError("a checkpoint needs H to be a multiple of 32")
        return Checkpoint(x.new_empty((T, H), dtype=torch.uint8),
                          x.new_empty((T, H // 32), dtype=torch.uint8), format)

    def _abi(self, T: int, H: int, device: int) -> _lib.Checkpoint:
        if self.format not in _lib.CHECKPOINTS:
            raise ValueError(f"format must be one of {sorted(_lib.CHECKPOINTS)}")
        return _lib.Checkpoint(_tensor(self.codes, "codes", (T, H), _U8, device),
                               _tensor(self.scales, "scales", (T, H // 32), _U8, device),
                               _lib.CHECKPOINTS[self.format])


def _rows_shape(x):
    t = x.codes if isinstance(x, Checkpoint) else x
    if t.dim() != 2:
        raise ValueError("rows must be [T, H]")
    T, H = t.shape
    if T >= 2 ** 31 or H >= 2 ** 31:
        _int32(T=T, H=H)
    return T, H, t


def _format(dtype: torch.dtype) -> int:
    if dtype not in _ROWS:
        raise TypeError(f"expected bf16 or fp32, not {dtype}")
    return _lib.ROWS_FP32 if dtype == torch.float32 else _lib.ROWS_BF16


def checkpoint_pack(x: torch.Tensor, format: str = "e4m3", out: Checkpoint | None = None,
                    stream=None) -> Checkpoint:
    """Rows [T, H] (bf16 or fp32, H a multiple of 32) stored in 8 bits, in `format`, or in `out` and
    its format."""
    if stream is None and out is None:
        done = _edge.checkpoint_pack(x, format)
        if done is not None:
            return Checkpoint(*done, format)
    T, H, t = _rows_shape(x)
    where = _elsewhere(t, stream)
    if where is not None:
        with where:
            return checkpoint_pack(x, format, out)
    dev = t.get_device()
    x = _aligned(x)
    xp = _tensor(x, "x", (T, H), _ROWS, dev)
    if out is None:
        out = Checkpoint._beside(x, format)
    check(lib.mxfp4_moe_checkpoint_pack(T, H, _format(x.dtype), xp, out._abi(T, H, dev),
                                        _current(dev)), "mxfp4_moe_checkpoint_pack")
    return out


def checkpoint_unpack(checkpoint: Checkpoint, dtype: torch.dtype = torch.bfloat16,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The rows [T, H] that a checkpoint stands for, as bf16 or fp32."""
    if stream is None and out is None and dtype in _ROWS:
        done = _edge.checkpoint_unpack(checkpoint.codes, checkpoint.scales, checkpoint.format,
                                       dtype == torch.float32)
        if done is not None:
            return done
    T, H, t = _rows_shape(checkpoint)
    where = _elsewhere(t, stream)
    if where is not None:
        with where:
            return checkpoint_unpack(checkpoint, dtype, out)
    dev = t.get_device()
    fmt = _format(dtype)
    frm = checkpoint._abi(T, H, dev)
    if out is None:
        out = t.new_empty((T, H), dtype=dtype)
        op = out.data_ptr() or _EMPTY
    else:
        op = _tensor(out, "out", (T, H), (dtype,), dev)
    check(lib.mxfp4_moe_checkpoint_unpack(T, H, fmt, frm, op, _current(dev)),
          "mxfp4_moe_checkpoint_unpack")
    return out


class NormOut(NamedTuple):
    out: torch.Tensor
    x_out: torch.Tensor | None          # x + y, where y was given
    mean: torch.Tensor | None           # fp32 [T]; None for "rms"
    rstd: torch.Tensor                  # fp32 [T]
    checkpoint: Checkpoint | None       # where one was asked for


@lru_cache(maxsize=1024)  # the library only reads them
def _norm_dims(T, H, kind, eps, rows: torch.dtype, params: torch.dtype) -> _lib.Norm:
    if kind not in _lib.NORMS:
        raise ValueError(f"kind must be one of {sorted(_lib.NORMS)}")
    return _lib.Norm(T, H, _lib.NORMS[kind], eps, _format(rows), _format(params))


@lru_cache(maxsize=1024)
def norm_workspace_bytes(T: int, H: int) -> int:
    """Scratch bytes of norm_backward with the parameters' gradients."""
    _int32(T=T, H=H)
    n = ctypes.c_size_t()
    check(lib.mxfp4_moe_norm_workspace_size(_lib.Norm(T, H, 0, 0.0, 0, 0), n),
          "mxfp4_moe_norm_workspace_size")
    return n.value


def norm_forward(x: torch.Tensor | Checkpoint, weight: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None, *, kind: str = "layer", eps: float = 1e-5,
                 y: torch.Tensor | None = None, checkpoint: str | Checkpoint | None = None,
                 dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                 x_out: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                 rstd: torch.Tensor | None = None, stream=None) -> NormOut:
    """Layer norm (kind "layer") or rms norm ("rms") of rows [T, H] in one kernel.

    x: bf16 or fp32 rows, or a Checkpoint (normalised as the rows it stands for, into `dtype`,
    bf16 by default).  y: a residual; x_out = x + y, rounded to the rows' type, is returned and
    is what is normalised.  checkpoint: a format or a Checkpoint to fill with those rows.  With a
    checkpoint, outputs that the caller gives begin at 16-byte addresses, and inputs that do not
    are copied first."""
    stored = isinstance(x, Checkpoint)
    if (stream is None and out is None and x_out is None and mean is None and rstd is None
            and not isinstance(checkpoint, Checkpoint)):
        done = None
        if not stored and dtype in (None, x.dtype):
            done = _edge.norm_forward(x, None, None, False, y, weight, bias, kind, eps, checkpoint)
        elif stored and y is None and checkpoint is None and dtype in (None, *_ROWS):
            done = _edge.norm_forward(x.codes, x.scales, x.format, dtype == torch.float32, None,
                                      weight, bias, kind, eps, None)
        if done is not None:
            kept = None if checkpoint is None else Checkpoint(done[4], done[5], checkpoint)
            return NormOut(*done[:4], kept)
    T, H, t = _rows_shape(x)
    if stored:
        if y is not None or checkpoint is not None:
            raise ValueError("a checkpoint as input takes no residual and fills no checkpoint")
        dtype = torch.bfloat16 if dtype is None else dtype
    elif dtype is not None and dtype != x.dtype:
        raise ValueError("dtype is the rows' own type, except for a checkpoint")
    else:
        dtype = x.dtype
    if y is None and x_out is not None:
        raise ValueError("x_out without a residual")
    params = dtype
    if weight is not None:
        params = weight.dtype
        if bias is not None and bias.dtype != params:
            raise TypeError("weight and bias must have the same type")
    elif bias is not None:
        params = bias.dtype
    dims = _norm_dims(T, H, kind, eps, dtype, params)
    where = _elsewhere(t, stream)
    if where is not None:
        with where:
            return norm_forward(x, weight, bias, kind=kind, eps=eps, y=y, checkpoint=checkpoint,
                                dtype=dtype, out=out, x_out=x_out, mean=mean, rstd=rstd)
    dev = t.get_device()
    rows, own = (T, H), (dtype,)
    xp = frm = yp = op = mp = to = None
    if stored or checkpoint is not None:
        x = x if stored else _aligned(x)
        y, weight, bias = _aligned(y), _aligned(weight), _aligned(bias)
    if stored:
        frm = x._abi(T, H, dev)
    else:
        xp = _tensor(x, "x", rows, own, dev)
    wp = None if weight is None else _tensor(weight, "weight", (H,), _ROWS, dev)
    bp = None if bias is None else _tensor(bias, "bias", (H,), _ROWS, dev)
    if y is not None:
        yp = _tensor(y, "y", rows, own, dev)
        if x_out is None:
            x_out = torch.empty_like(x)
            op = x_out.data_ptr() or _EMPTY
        else:
            op = _tensor(x_out, "x_out", rows, own, dev)
    if checkpoint is not None:
        if not isinstance(checkpoint, Checkpoint):
            checkpoint = Checkpoint._beside(x, checkpoint)
        to = checkpoint._abi(T, H, dev)
    if out is None:
        out = t.new_empty(rows, dtype=dtype) if stored else torch.empty_like(x)
        np_ = out.data_ptr() or _EMPTY
    else:
        np_ = _tensor(out, "out", rows, own, dev)
    if rstd is None:
        rstd = t.new_empty(T, dtype=torch.float32)
        rp = rstd.data_ptr() or _EMPTY
    else:
        rp = _tensor(rstd, "rstd", (T,), _F32, dev)
    if mean is not None:
        mp = _tensor(mean, "mean", (T,), _F32, dev)
    elif kind == "layer":
        mean = torch.empty_like(rstd)
        mp = mean.data_ptr() or _EMPTY
    check(lib.mxfp4_moe_norm_forward(dims, xp, frm, yp, wp, bp, op, to, np_, mp, rp,
                                     _current(dev)), "mxfp4_moe_norm_forward")
    return NormOut(out, x_out, mean, rstd, checkpoint)


def norm_backward(d_out: torch.Tensor, x: torch.Tensor | Checkpoint, mean: torch.Tensor | None,
                  rstd: torch.Tensor, weight: torch.Tensor | None = None, *, kind: str = "layer",
                  g: torch.Tensor | None = None, params: bool = True,
                  dx: torch.Tensor | None = None, d_weight: torch.Tensor | None = None,
                  d_bias: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                  stream=None):
    """(dx [+ g], d_weight, d_bias) of `norm_forward`; the parameters' gradients are fp32 [H].

    x: the rows that were normalised (x_out where a residual was added), or their checkpoint with
    the statistics of the forward on it.  g: the residual stream's gradient, added to dx (dx may
    be g itself).  params=False computes dx alone and returns None for the other two; d_bias is
    None for "rms" unless a tensor is given.  With a checkpoint, dx begins at a 16-byte address, and
    inputs that do not are copied first.  ws: scratch of norm_workspace_bytes (else
    allocated); two captured graphs that may run at once need one each."""
    if (stream is None and params and dx is None and d_weight is None and d_bias is None
            and ws is None):
        done = (_edge.norm_backward(d_out, x.codes, x.scales, x.format, mean, rstd, weight, kind, g)
                if isinstance(x, Checkpoint) else
                _edge.norm_backward(d_out, x, None, None, mean, rstd, weight, kind, g))
        if done is not None:
            return done
    T, H, t = _rows_shape(x)
    dtype = d_out.dtype
    dims = _norm_dims(T, H, kind, 0.0, dtype, dtype if weight is None else weight.dtype)
    if kind == "layer" and mean is None:
        raise ValueError("the layer norm's backward needs the mean")
    if not params and (d_weight is not None or d_bias is not None):
        raise ValueError("params=False with an output for the parameters' gradient")
    where = _elsewhere(t, stream)
    if where is not None:
        with where:
            return norm_backward(d_out, x, mean, rstd, weight, kind=kind, g=g, params=params,
                                 dx=dx, d_weight=d_weight, d_bias=d_bias, ws=ws)
    dev = t.get_device()
    rows, own = (T, H), (dtype,)
    xp = frm = dwp = dbp = wsp = None
    if isinstance(x, Checkpoint):
        d_out, weight, g = _aligned(d_out), _aligned(weight), g if g is dx else _aligned(g)
    dp = _tensor(d_out, "d_out", rows, _ROWS, dev)
    if isinstance(x, Checkpoint):
        frm = x._abi(T, H, dev)
    else:
        xp = _tensor(x, "x", rows, own, dev)
    mp = None if mean is None else _tensor(mean, "mean", (T,), _F32, dev)
    rp = _tensor(rstd, "rstd", (T,), _F32, dev)
    wp = None if weight is None else _tensor(weight, "weight", (H,), _ROWS, dev)
    gp = None if g is None else _tensor(g, "g", rows, own, dev)
    if dx is None:
        dx = torch.empty_like(d_out)
        op = dx.data_ptr() or _EMPTY
    else:
        op = _tensor(dx, "dx", rows, own, dev)
    ws_bytes = 0
    if params:
        if d_weight is None:
            d_weight = rstd.new_empty(H)
            dwp = d_weight.data_ptr()
        else:
            dwp = _tensor(d_weight, "d_weight", (H,), _F32, dev)
        if d_bias is not None:
            dbp = _tensor(d_bias, "d_bias", (H,), _F32, dev)
        elif kind == "layer":
            d_bias = torch.empty_like(d_weight)
            dbp = d_bias.data_ptr()
        if ws is None:
            ws_bytes = norm_workspace_bytes(T, H)
            ws = t.new_empty(ws_bytes, dtype=torch.uint8)
        elif ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous, on cuda:{dev}")
        else:
            ws_bytes = ws.numel() * ws.element_size()
        wsp = ws.data_ptr() or None
    check(lib.mxfp4_moe_norm_backward(dims, dp, xp, frm, mp, rp, wp, gp, op, dwp, dbp, wsp,
                                      ws_bytes, _current(dev)), "mxfp4_moe_norm_backward")
    return dx, d_weight, d_bias


def selftest_wait_timeout(ws: torch.Tensor, stream=None) -> None:
    """Enqueue the failure-detection self-test on `ws` (first 16 bytes zero); read the outcome
    with device_check(ws): (MXFP4_MOE_ERR_DEVICE_TIMEOUT, 0xF00) after about one second."""
    check(lib.mxfp4_moe_selftest_wait_timeout(_ptr(ws), ws.numel() * ws.element_size(),
                                               _stream(stream)), "mxfp4_moe_selftest_wait_timeout")


def weights_to(inp: dict, device) -> dict:
    keys = ("gu_blocks", "gu_scales", "gu_bias", "dn_blocks", "dn_scales", "dn_bias")
    return {k: inp[k].to(device).contiguous() for k in keys}


def profile_begin() -> None:
    check(lib.mxfp4_moe_profile_begin(), "mxfp4_moe_profile_begin")


def profile_end() -> dict:
    """{kernel name: (launches, total device ms)} since profile_begin()."""
    buf = (_lib.KernelTime * 64)()
    n = ctypes.c_int32(0)
    check(lib.mxfp4_moe_profile_end(buf, 64, ctypes.byref(n)), "mxfp4_moe_profile_end")
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n.value)}
