"""AdamW over a list of tensors, with the moments in fp32 or in 8 bits.

    p = plan(weights, grads, copies=[layer's bf16 weights], bits=8, weight_decay=0.1)
    step(p, lr=3e-4, step=t)            # t = 1, 2, ...

The weights are fp32 masters; `copies` (each or any None) get them rounded to bf16, which is
what the layer computes with.  A plan holds its tensors: gradients are read from the ones it
was made with.  The step is one launch for up to 96 tensors (moe_adamw_* of include/moe.h,
where the formulas and the 8-bit format are).
"""
from __future__ import annotations

import array
import ctypes
from dataclasses import dataclass
from typing import List, Optional

import torch

from . import binding as B

BLOCK = 128     # elements that share a scale in the 8-bit states


@dataclass
class Plan:
    weights: List[torch.Tensor]
    grads: List[torch.Tensor]
    copies: List[Optional[torch.Tensor]]
    m: List[torch.Tensor]
    v: List[torch.Tensor]
    m_scale: Optional[List[torch.Tensor]]
    v_scale: Optional[List[torch.Tensor]]
    bits: int
    table: ctypes.Array         # the entry point's descriptors of the above
    hyper: B.moe_adamw_hyper
    device: torch.device
    shapes: List[torch.Size]    # of the weights

    def check_device(self, stream=None):
        B.check_device(self.device, stream)


def plan(weights, grads, copies=None, bits=32, weight_decay=0.0, m=None, v=None, m_scale=None, v_scale=None) -> Plan:
    """weights: fp32; grads: bf16 or fp32; copies: bf16 or None; weight_decay: one number or one a tensor.  The
    states start at zero, or are the ones given (a resumed run's): fp32, or int8 / uint8 codes with their scales
    [ceil(n / 128)]."""
    if bits not in (32, 8):
        raise ValueError("bits: 32 or 8")
    weights, grads = list(weights), list(grads)
    n = len(weights)
    copies = [None] * n if copies is None else list(copies)
    decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
    kinds = (torch.float32, torch.float32) if bits == 32 else (torch.int8, torch.uint8)
    fresh = lambda kind: [torch.zeros(w.shape, dtype=kind, device=w.device) for w in weights]  # noqa: E731
    blocks = [(-(-w.numel() // BLOCK),) for w in weights]
    scales = lambda: [torch.zeros(b, device=w.device) for b, w in zip(blocks, weights)]  # noqa: E731
    m, v = fresh(kinds[0]) if m is None else list(m), fresh(kinds[1]) if v is None else list(v)
    if bits == 8:
        m_scale = scales() if m_scale is None else list(m_scale)
        v_scale = scales() if v_scale is None else list(v_scale)
    elif m_scale is not None or v_scale is not None:
        raise ValueError("scales belong to 8-bit states")
    every = [weights, grads, copies, decay, m, v] + ([m_scale, v_scale] if bits == 8 else [])
    if any(len(x) != n for x in every):
        raise ValueError("as many gradients, copies, decays and states as weights")
    if any(t is None for x in every if x is not copies for t in x):
        raise ValueError("only copies may be None")
    device = weights[0].device if n else torch.device("cuda")
    if any(w.device != device for w in weights):
        raise ValueError("weights on more than one device")
    table = (B.moe_adamw_tensor * max(1, n))()
    for i, w in enumerate(weights):
        B.check_tensor(w, torch.float32, w.shape, w.device)
        B.check_tensor(grads[i], torch.bfloat16 if grads[i].dtype == torch.bfloat16 else torch.float32, w.shape, w.device)
        B.check_tensor(copies[i], torch.bfloat16, w.shape, w.device)
        B.check_tensor(m[i], kinds[0], w.shape, w.device)
        B.check_tensor(v[i], kinds[1], w.shape, w.device)
        t = table[i]
        if bits == 8:
            B.check_tensor(m_scale[i], torch.float32, blocks[i], w.device)
            B.check_tensor(v_scale[i], torch.float32, blocks[i], w.device)
            t.m_scale, t.v_scale = m_scale[i].data_ptr(), v_scale[i].data_ptr()
        t.w, t.grad, t.m, t.v = (x.data_ptr() for x in (w, grads[i], m[i], v[i]))
        t.w16 = None if copies[i] is None else copies[i].data_ptr()
        t.n, t.weight_decay = w.numel(), decay[i]
        t.grad_type = B.TYPE["bf16" if grads[i].dtype == torch.bfloat16 else "fp32"]
    return Plan(weights, grads, copies, m, v, m_scale, v_scale, bits, table, B.moe_adamw_hyper(bits=bits), device,
                [w.shape for w in weights])


def step(p: Plan, lr, step, beta1=0.9, beta2=0.95, eps=1e-8, seed=0, control=None, stream=None):
    """Updates p's weights, copies and states.  seed: of the 8-bit states' draws.  control: a Control, whose values
    on the device then take the place of `step` and scale lr and the gradients (for captured steps).  eps: above 0
    in fp32, and at least 2^-63 with 8-bit states."""
    p.check_device(stream)
    if control is not None and p.weights:
        B.check_tensor(control.raw, torch.int32, (4,), p.device)
    h = p.hyper
    h.lr, h.beta1, h.beta2, h.eps, h.step, h.seed = lr, beta1, beta2, eps, step, seed
    B.moe_adamw_step(h, p.table, len(p.weights), None if control is None else control.raw, stream)


class Control:
    """What a step takes from device memory: one-element views to write to, on the stream of the step."""

    def __init__(self, device="cuda"):
        self.raw = torch.zeros(4, dtype=torch.int32, device=device)
        self.grad_scale, self.lr_scale = self.raw.view(torch.float32)[0:1], self.raw.view(torch.float32)[1:2]
        self.step, self.skip = self.raw[2:3], self.raw[3:4]
        self.grad_scale.fill_(1.0)
        self.lr_scale.fill_(1.0)
        self.step.fill_(1)


def values(p: Plan, m_out=None, v_out=None, dtype=torch.bfloat16, stream=None):
    """The moments that p's 8-bit states stand for, as lists of tensors (new ones of `dtype`, or the given)."""
    if p.bits != 8:
        raise ValueError("values: the states are held in fp32 as they are")
    p.check_device(stream)
    new = lambda: [torch.empty(s, dtype=dtype, device=p.device) for s in p.shapes]  # noqa: E731
    m_out, v_out = new() if m_out is None else list(m_out), new() if v_out is None else list(v_out)
    kind = m_out[0].dtype if m_out else dtype
    if kind not in (torch.bfloat16, torch.float32):
        raise ValueError("values: bf16 or fp32 tensors")
    B.check_tensors(m_out, kind, p.shapes, p.device)
    B.check_tensors(v_out, kind, p.shapes, p.device)
    pointers = lambda ts: (ctypes.c_void_p * max(1, len(ts))).from_buffer(  # noqa: E731
        array.array("Q", [t.data_ptr() for t in ts] or [0]))
    B.moe_adamw_values(p.table, len(p.weights), B.TYPE["bf16" if kind == torch.bfloat16 else "fp32"], pointers(m_out),
                       pointers(v_out), stream)
    return m_out, v_out
