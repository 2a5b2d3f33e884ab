"""The norms around a block and the merge of its output into the residual stream.

    x = norm(h)                                  norm_forward: the block's input
    h_out = alpha h + beta gate norm(y)          merge_forward: y is the block's output
    x_next = norm(h_out)                         ... with w_next: the next block's input

PyTorch only allocates; every step runs in libmoe.so's kernels (moe_norm_*, moe_merge_* of
include/moe.h, where the formulas are).  One `Buffers` serves one norm or merge of a block;
its outputs are overwritten by the next call.  It holds the outputs of either direction of
both: 16384 x 7168 bf16 take 0.95 GB, of which a norm's forward writes a quarter.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as B

_DTYPE = {B.TYPE["bf16"]: torch.bfloat16, B.TYPE["fp32"]: torch.float32}


@dataclass
class Buffers:
    dims: B.moe_norm_dims
    h_out: torch.Tensor        # [T, d] the stream after the merge
    x: torch.Tensor            # [T, d] bf16 the norm's output
    dh: torch.Tensor           # [T, d] gradient of the stream
    dy: torch.Tensor           # [T, d] bf16 gradient of the block's output
    dw: torch.Tensor           # [d] fp32 gradient of the norm's weight (merge: of w_next)
    dw_post: torch.Tensor      # [d] fp32
    dgate: Optional[torch.Tensor]  # [d] or [T] fp32
    workspace: torch.Tensor


def dims_of(T, d, stream="bf16", weights="fp32", gate="none", gate_act="identity", eps=1e-6, weight_offset=0.0,
            alpha=1.0, beta=1.0) -> B.moe_norm_dims:
    """stream, weights: "bf16" or "fp32"; gate: "none", "channel" ([d] of the weights' type) or "token"
    ([T] fp32); gate_act: "identity" or "sigmoid"."""
    dims = B.make_norm_dims(T, d, stream, weights, gate, gate_act, eps, weight_offset, alpha, beta)
    st = B.moe_norm_check_dims(dims)
    if st != B.MOE_OK:
        raise B.MoeError("moe_norm_check_dims", st)
    return dims


def allocate(dims: B.moe_norm_dims, device="cuda") -> Buffers:
    T, d, stream = dims.T, dims.d, _DTYPE[dims.stream_type]
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
    gate = None if dims.gate == B.GATE["none"] else e(d if dims.gate == B.GATE["channel"] else T)
    return Buffers(dims=dims, h_out=e(T, d, dt=stream), x=e(T, d, dt=torch.bfloat16), dh=e(T, d, dt=stream),
                   dy=e(T, d, dt=torch.bfloat16), dw=e(d), dw_post=e(d), dgate=gate,
                   workspace=e(B.moe_norm_workspace_size(dims), dt=torch.uint8))


def _check(b: Buffers, on, stream=(), block=(), weights=(), gate=None):
    """Rows of the residual stream, rows of the block and weights as the call's dims have them, on the device that a
    call with the CUDA stream `on` runs on."""
    dm, dev = b.dims, b.x.device
    B.check_device(dev, on)
    rows, n = (dm.T, dm.d), (dm.d,)
    for t in stream:
        B.check_tensor(t, _DTYPE[dm.stream_type], rows, dev)
    for t in block:
        B.check_tensor(t, torch.bfloat16, rows, dev)
    for t in weights:
        B.check_tensor(t, _DTYPE[dm.weight_type], n, dev)
    if gate is not None:
        if dm.gate == B.GATE["token"]:
            B.check_tensor(gate, torch.float32, (dm.T,), dev)
        else:
            B.check_tensor(gate, _DTYPE[dm.weight_type], n, dev)


def norm_forward(b: Buffers, h, w, stream=None):
    """-> b.x"""
    _check(b, stream, stream=(h,), weights=(w,))
    B.moe_norm_fwd(b.dims, h, w, b.x, stream)
    return b.x


def norm_backward(b: Buffers, dx, h, w, dh_add=None, stream=None):
    """-> b.dh (dh_add, the gradient that reaches h around the block, added to it) and b.dw."""
    _check(b, stream, stream=(h, dh_add), block=(dx,), weights=(w,))
    B.moe_norm_bwd(b.dims, dx, h, w, dh_add, b.dh, b.dw, b.workspace, stream)
    return b.dh


def merge_forward(b: Buffers, h, y, w_post=None, gate=None, w_next=None, stream=None):
    """-> b.h_out, and b.x (the next block's input) where w_next is given."""
    _check(b, stream, stream=(h,), block=(y,), weights=(w_post, w_next), gate=gate)
    B.moe_merge_fwd(b.dims, h, y, w_post, gate, w_next, b.h_out, None if w_next is None else b.x, stream)
    return b.h_out


def merge_backward(b: Buffers, dh_out, dx_next, h_out, y, w_post=None, gate=None, w_next=None, stream=None):
    """-> b.dh, b.dy and the gradients of what is given: b.dw_post, b.dgate, b.dw (of w_next).  dh_out (the
    gradient of h_out) may be None where w_next is given, dx_next (of b.x) is None where it is not."""
    _check(b, stream, stream=(dh_out, h_out), block=(dx_next, y), weights=(w_post, w_next), gate=gate)
    B.moe_merge_bwd(b.dims, dh_out, dx_next, h_out, y, w_post, gate, w_next, b.dh, b.dy,
                    None if w_post is None else b.dw_post, b.dgate, None if w_next is None else b.dw, b.workspace,
                    stream)
    return b.dh
