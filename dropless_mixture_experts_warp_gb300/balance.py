"""The router's balance loss, z-loss and per-expert counts over ragged sequences.

forward() after moe_route_topk (it takes the same logits and topk_idx), backward() after
moe_route_topk_bwd, to whose d_logits it adds.  PyTorch only allocates; the steps run in
libmoe.so's kernels (moe_balance_* of include/moe.h, where the formulas are).
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B


@dataclass
class Buffers:
    dims: B.moe_balance_dims
    losses: torch.Tensor       # [2] fp32: balance loss, z-loss
    counts: torch.Tensor       # [sequences, E] int32
    prob_mean: torch.Tensor    # [sequences, E] fp32
    seq_tokens: torch.Tensor   # [sequences] int32
    workspace: torch.Tensor
    status: torch.Tensor


def allocate(T, E, k, score="softmax", sequences=1, device="cuda") -> Buffers:
    dims = B.make_balance_dims(T, E, k, score, sequences)
    st = B.moe_balance_check_dims(dims)
    if st != B.MOE_OK:
        raise B.MoeError("moe_balance_check_dims", st)
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
    return Buffers(dims=dims, losses=e(2), counts=e(sequences, E, dt=torch.int32), prob_mean=e(sequences, E),
                   seq_tokens=e(sequences, dt=torch.int32),
                   workspace=e(B.moe_balance_workspace_size(dims), dt=torch.uint8),
                   status=torch.zeros(1, dtype=torch.int32, device=device))


def _inputs(b: Buffers, on, logits, seq_offsets, mask):
    dm, dev = b.dims, b.losses.device
    B.check_device(dev, on)
    B.check_tensor(logits, torch.float32, (dm.T, dm.E), dev)
    B.check_tensor(seq_offsets, torch.int32, (dm.S + 1,), dev)
    B.check_tensor(mask, torch.uint8, (dm.T,), dev)


def forward(b: Buffers, logits, topk_idx, seq_offsets=None, mask=None, coef=1.0, z_coef=0.0, stream=None):
    """-> b.losses (coef and z_coef included); also b.counts, b.prob_mean, b.seq_tokens.  seq_offsets
    [sequences + 1] int32 (None: one sequence), mask [T] uint8, 0 = padding (None: no padding)."""
    _inputs(b, stream, logits, seq_offsets, mask)
    B.check_tensor(topk_idx, torch.int32, (b.dims.T, b.dims.k), b.losses.device)
    b.dims.coef, b.dims.z_coef = coef, z_coef
    B.moe_balance_fwd(b.dims, logits, topk_idx, seq_offsets, mask, b.losses, b.counts, b.prob_mean, b.seq_tokens,
                      b.workspace, b.status, stream)
    return b.losses


def backward(b: Buffers, logits, d_logits, seq_offsets=None, mask=None, coef=None, z_coef=None, grad=None,
             accumulate=True, stream=None):
    """Adds to d_logits [T, E] (accumulate=False: writes) the gradient of grad[0] * losses[0] + grad[1] *
    losses[1] (grad [2] fp32 on the device; None: 1, 1), from the counts that forward() left in b.  coef, z_coef:
    None takes those of b's last forward(), whose losses these are; others count for this call alone."""
    _inputs(b, stream, logits, seq_offsets, mask)
    dims = b.dims
    if coef is not None or z_coef is not None:
        dims = type(dims).from_buffer_copy(dims)
        dims.coef, dims.z_coef = (own if given is None else given for given, own in ((coef, dims.coef), (z_coef, dims.z_coef)))
    B.check_tensor(d_logits, torch.float32, (b.dims.T, b.dims.E), b.losses.device)
    B.check_tensor(grad, torch.float32, (2,), b.losses.device)
    B.moe_balance_bwd(dims, logits, seq_offsets, mask, b.counts, b.seq_tokens, grad, accumulate, d_logits, stream)
    return d_logits


def check(b: Buffers, stream=None):
    """Raise on a device-side error (an expert index or sequence offsets out of range)."""
    st = B.moe_check_status(b.status, stream)
    if st != B.MOE_OK:
        raise B.MoeError("device status", st)
