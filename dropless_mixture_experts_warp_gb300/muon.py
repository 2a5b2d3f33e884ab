"""Steps along orthogonalised updates (Muon) over a list of matrices, beside optim.py's AdamW.

    p = plan(weights, grads, copies=[layer's bf16 weights], weight_decay=0.1)
    step(p, lr=2e-4)

Every tensor is a matrix [m, n] or a batch of them [..., m, n] (an expert weight [E, 2f, d] holds a gate and an up
matrix: pass its view(2 * E, f, d)).  The momentum is orthogonalised by Newton-Schulz products and taken off the fp32
weights; `copies` (each or any None) get them rounded to bf16.  orthogonalize() does that alone.  The products are as good
as fp32's (operands in two fp16 parts), or with products="fp16" take a third of the multiplying and leave the orthogonal
factor some 1e-3 off (include/moe.h says how far), a step's fp32 weights some 1e-6.  The steps run in
libmoe.so's kernels (moe_muon_* of include/moe.h, where the formulas are); norms, routers' biases and other vectors
are optim.py's.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import List, Optional

import torch

from . import binding as B

COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5     # a, b, c of each Newton-Schulz step
WORKSPACE = 8 << 30                                 # bytes at most, unless one matrix needs more


@dataclass
class Plan:
    weights: List[torch.Tensor]
    grads: List[torch.Tensor]
    copies: List[Optional[torch.Tensor]]
    m: List[torch.Tensor]
    table: ctypes.Array          # the entry point's descriptors of the above
    workspace: torch.Tensor
    status: torch.Tensor
    hyper: B.moe_muon_hyper
    device: torch.device
    products: int


@dataclass
class Workspace:
    shapes: List[torch.Size]
    table: ctypes.Array
    workspace: torch.Tensor
    status: torch.Tensor
    hyper: B.moe_muon_hyper
    device: torch.device
    products: int


def _sides(shape):
    if len(shape) < 2:
        raise ValueError(f"matrices or batches of them: got {tuple(shape)}")
    batch = 1
    for s in shape[:-2]:
        batch *= s
    return batch, shape[-2], shape[-1]


def _apart(spans):
    """Refuse memory that is written and shared: the matrices of a call run in no order.  spans: (start, stop, written)."""
    end = end_written = 0
    for start, stop, written in sorted(spans):
        if start < (end if written else end_written) and start < stop:
            raise ValueError("a tensor that is written shares memory with another of the call")
        if stop > end:
            end = stop
        if written and stop > end_written:
            end_written = stop


def _span(t, written):
    at = t.data_ptr()
    return at, at + t.numel() * t.element_size(), written


def _hyper(lr, momentum, rms, nesterov, coefficients):
    coefficients = [tuple(c) for c in coefficients]
    if not 1 <= len(coefficients) <= B.MUON_MAX_STEPS or any(len(c) != 3 for c in coefficients):
        raise ValueError(f"coefficients: a, b, c of 1 to {B.MUON_MAX_STEPS} steps")
    h = B.moe_muon_hyper(lr=lr, momentum=momentum, rms=rms, nesterov=int(nesterov), steps=len(coefficients))
    h.coefficients[:3 * len(coefficients)] = [x for c in coefficients for x in c]
    return h


def _products(name):
    if name not in B.MUON_PRODUCTS:
        raise ValueError('products: "fp32" or "fp16"')
    return B.MUON_PRODUCTS[name]


def _allocate(table, n, limit, device, products):
    return (torch.empty(max(16, B.moe_muon_workspace_size_with(table, n, limit, products)), dtype=torch.uint8, device=device),
            torch.zeros(1, dtype=torch.int32, device=device))


def plan(weights, grads, copies=None, weight_decay=0.0, m=None, coefficients=COEFFICIENTS, workspace=WORKSPACE,
         products="fp32") -> Plan:
    """weights: fp32; grads: bf16 or fp32; copies: bf16 or None; weight_decay: one number or one a tensor.  The
    momentum starts at zero, or is the one given (a resumed run's, fp32).  No tensor may share memory with another, but
    gradients with each other.  workspace: bytes of scratch at most; a plan's
    steps share it, so they follow one another, also as replays of captured graphs."""
    weights, grads = list(weights), list(grads)
    n = len(weights)
    copies = [None] * n if copies is None else list(copies)
    decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
    m = [torch.zeros_like(w) for w in weights] if m is None else list(m)
    if any(len(x) != n for x in (grads, copies, decay, m)):
        raise ValueError("as many gradients, copies, decays and momenta as weights")
    if any(t is None for x in (weights, grads, decay, m) for t in x):
        raise ValueError("only copies may be None")
    device = weights[0].device if n else torch.device("cuda")
    if any(w.device != device for w in weights):
        raise ValueError("weights on more than one device")
    if any(len({t.data_ptr() for t in x if t.numel()}) < sum(t.numel() > 0 for t in x) for x in (weights, m)):
        raise ValueError("a tensor is in the list twice")
    table = (B.moe_muon_tensor * max(1, n))()
    for i, w in enumerate(weights):
        low = grads[i].dtype == torch.bfloat16
        B.check_tensor(w, torch.float32, w.shape, device)
        B.check_tensor(grads[i], torch.bfloat16 if low else torch.float32, w.shape, device)
        B.check_tensor(copies[i], torch.bfloat16, w.shape, device)
        B.check_tensor(m[i], torch.float32, w.shape, device)
        t = table[i]
        t.batch, t.rows, t.cols = _sides(w.shape)
        t.grad, t.m, t.w = grads[i].data_ptr(), m[i].data_ptr(), w.data_ptr()
        t.w16 = None if copies[i] is None else copies[i].data_ptr()
        t.weight_decay, t.grad_type = decay[i], B.TYPE["bf16" if low else "fp32"]
    _apart([_span(t, True) for t in weights + m + copies if t is not None] + [_span(t, False) for t in grads])
    kind = _products(products)
    return Plan(weights, grads, copies, m, table, *_allocate(table, n, workspace, device, kind),
                _hyper(0.0, 0.0, 0.0, True, coefficients), device, kind)


def step(p: Plan, lr, momentum=0.95, rms=0.2, nesterov=True, control=None, stream=None, eps=1e-7):
    """Updates p's momenta, weights and copies.  rms: root mean square of the update's elements at lr = 1 (of a full
    orthogonal factor).  control: an optim.Control, whose scales and skip the kernels then read on the device.  eps:
    a matrix whose update's norm is below it is divided by eps instead, so that the steps of an expert without tokens fade
    with its momentum (0: every matrix that is not 0 takes full steps)."""
    B.check_device(p.device, stream)
    raw = None if control is None else control.raw
    if p.weights:
        B.check_tensor(raw, torch.int32, (4,), p.device)
    h = p.hyper
    h.lr, h.momentum, h.rms, h.nesterov = lr, momentum, rms, int(nesterov)
    B.moe_muon_step_with(h, p.table, len(p.weights), eps, p.products, p.workspace, p.workspace.numel(), raw, p.status, stream)


def workspace(shapes, coefficients=COEFFICIENTS, limit=WORKSPACE, device="cuda", products="fp32") -> Workspace:
    """What orthogonalize() needs for tensors of these shapes, and how it multiplies."""
    shapes = [torch.Size(s) for s in shapes]
    table = (B.moe_muon_tensor * max(1, len(shapes)))()
    for t, s in zip(table, shapes):
        t.batch, t.rows, t.cols = _sides(s)
    kind = _products(products)
    ws, status = _allocate(table, len(shapes), limit, device, kind)
    return Workspace(shapes, table, ws, status, _hyper(0.0, 0.0, 0.0, False, coefficients), ws.device, kind)


def orthogonalize(xs, outs, w: Workspace, stream=None):
    """outs[i] (bf16 or fp32) = the orthogonal factor of xs[i] (bf16 or fp32) as the steps approximate it.  outs[i] may be
    xs[i] itself; no output may share memory otherwise."""
    B.check_device(w.device, stream)
    if len(xs) != len(w.shapes) or len(outs) != len(w.shapes):
        raise ValueError(f"expected {len(w.shapes)} tensors, got {len(xs)} and {len(outs)}")
    spans = []
    for t, s, x, o in zip(w.table, w.shapes, xs, outs):
        kind = [torch.bfloat16 if y.dtype == torch.bfloat16 else torch.float32 for y in (x, o)]
        B.check_tensor(x, kind[0], s, w.device)
        B.check_tensor(o, kind[1], s, w.device)
        t.grad, t.out = x.data_ptr(), o.data_ptr()
        t.grad_type, t.out_type = (B.TYPE["bf16" if k == torch.bfloat16 else "fp32"] for k in kind)
        spans.append(_span(o, True))
        if t.grad != t.out or t.grad_type != t.out_type:
            spans.append(_span(x, False))
    _apart(spans)
    B.moe_muon_step_with(w.hyper, w.table, len(xs), 0.0, w.products, w.workspace, w.workspace.numel(), None, w.status, stream)
    return outs


def check(p, stream=None):
    """Raise on an error that a step of p (a Plan or a Workspace) found on the device."""
    st = B.moe_check_status(p.status, stream)
    if st != B.MOE_OK:
        raise B.MoeError("device status", st)
