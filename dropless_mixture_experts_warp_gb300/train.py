"""A stack of MoE blocks trained end to end: norms, router, balance loss, MoE layer, merge, AdamW or Muon.

    x_0 = norm(h_0)                                    moe_norm_fwd
    y_i = MoE layer(x_i, logits = x_i W_r^T)           layer.forward; balance.forward on its routing
    h_{i+1} = h_i + gate_i norm(y_i);  x_{i+1} = norm(h_{i+1})          moe_merge_fwd, one pass
    loss = mean (x_L - target)^2 + sum of the blocks' balance and z-losses

The gradient is the chain of the backward calls; the update is one optim.step over every weight, or with
optimizer="muon" one muon.step over the expert and router matrices and one optim.step over the rest.  The router's
projection (logits, its gradients) is a library GEMM in fp32, outside the layer as everywhere in this package.

    python -m dropless_mixture_experts_warp_gb300.train --steps 30 --bits 8
    python -m dropless_mixture_experts_warp_gb300.train --steps 30 --optimizer muon --prec fp8-block
"""
from __future__ import annotations

import argparse
import math
from typing import Optional

import torch

from . import balance, block, layer, muon, optim


class Stack:
    """L blocks of one shape for T tokens a step: weights, buffers and the calls of a step."""

    def __init__(self, T, d, f, E, k, blocks=2, score="softmax", stream="bf16", sequences=1, coef=1e-2, z_coef=1e-3,
                 bits=32, seed=0, device="cuda", prec="bf16", optimizer="adamw"):
        if optimizer not in ("adamw", "muon"):
            raise ValueError('optimizer: "adamw" or "muon"')
        self.T, self.L, self.coef, self.z_coef = T, blocks, coef, z_coef
        self.stream = torch.bfloat16 if stream == "bf16" else torch.float32
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda *s, fan: torch.randn(*s, generator=g, device=device) / math.sqrt(fan)  # noqa: E731
        dims = layer.dims_of(T, d, f, E, k, score=score, prec=prec)
        norm = block.dims_of(T, d, stream=stream, gate="channel")
        # norms[i] belongs to x_i: one before each block, one after the last
        self.norms = [torch.ones(d, device=device) for _ in range(blocks + 1)]
        self.blocks = [dict(router=rand(E, d, fan=d), gu=rand(E, 2 * f, d, fan=d), down=rand(E, d, f, fan=f),
                            post=torch.ones(d, device=device), gate=torch.full((d,), 0.5, device=device))
                       for _ in range(blocks)]
        self.low = [{n: b[n].bfloat16() for n in ("gu", "down")} for b in self.blocks]   # what the layer computes with
        self.pre = block.allocate(norm)
        self.bufs = [layer.allocate(dims) for _ in range(blocks)]
        self.merges = [block.allocate(norm) for _ in range(blocks)]
        self.balances = [balance.allocate(T, E, k, score=score, sequences=sequences) for _ in range(blocks)]
        self.d_router = [torch.empty(E, d, device=device) for _ in range(blocks)]
        self.logits = [None] * blocks
        weights, grads, copies, decay = [], [], [], []
        matrices = [], [], [], []                  # the same for Muon

        def add(w, grad, copy=None, wd=0.0):
            weights.append(w), grads.append(grad), copies.append(copy), decay.append(wd)

        def add_matrix(w, grad, copy=None, wd=0.0):
            if optimizer == "adamw":
                return add(w, grad, copy, wd)
            for to, x in zip(matrices, (w, grad, copy, wd)):
                to.append(x)

        halves = lambda x: x.view(2 * E, f, d)  # gate and up are matrices of their own  # noqa: E731
        for i, b in enumerate(self.blocks):
            add_matrix(halves(b["gu"]), halves(self.bufs[i].dw_gu), halves(self.low[i]["gu"]), 0.1)
            add_matrix(b["down"], self.bufs[i].dw_d, self.low[i]["down"], 0.1)
            add_matrix(b["router"], self.d_router[i], wd=0.1)
            add(b["post"], self.merges[i].dw_post)
            add(b["gate"], self.merges[i].dgate)
            add(self.norms[i], self.pre.dw if i == 0 else self.merges[i - 1].dw)
        add(self.norms[-1], self.merges[-1].dw)
        self.plan = optim.plan(weights, grads, copies=copies, bits=bits, weight_decay=decay)
        self.matrices = None
        if optimizer == "muon":
            self.matrices = muon.plan(matrices[0], matrices[1], copies=matrices[2], weight_decay=matrices[3])

    def forward(self, h, seq_offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None):
        """The stream h [T, d] -> x_L [T, d] bf16; the blocks' losses are in self.balances[i].losses."""
        self.h0, self.seqs, self.mask = h, seq_offsets, mask
        x = block.norm_forward(self.pre, h, self.norms[0])
        for i, b in enumerate(self.blocks):
            self.logits[i] = x.float() @ b["router"].t()
            y = layer.forward(self.bufs[i], x, self.logits[i], self.low[i]["gu"], self.low[i]["down"])
            balance.forward(self.balances[i], self.logits[i], self.bufs[i].topk_idx, seq_offsets=seq_offsets, mask=mask,
                            coef=self.coef, z_coef=self.z_coef)
            m = self.merges[i]
            h = block.merge_forward(m, h, y, w_post=b["post"], gate=b["gate"], w_next=self.norms[i + 1])
            x = m.x
        return x

    def backward(self, dx):
        """From the gradient of x_L (bf16) to every weight's; returns the gradient of h_0."""
        dh = None
        for i in reversed(range(self.L)):
            b, m, bufs = self.blocks[i], self.merges[i], self.bufs[i]
            dh = block.merge_backward(m, dh, dx, m.h_out, bufs.y, w_post=b["post"], gate=b["gate"],
                                      w_next=self.norms[i + 1])
            x = self.pre.x if i == 0 else self.merges[i - 1].x
            dxe = layer.backward(bufs, m.dy, self.logits[i], self.low[i]["gu"], self.low[i]["down"], x=x)
            dl = balance.backward(self.balances[i], self.logits[i], bufs.d_logits, seq_offsets=self.seqs, mask=self.mask,
                                  coef=self.coef, z_coef=self.z_coef)
            torch.mm(dl.t(), x.float(), out=self.d_router[i])
            dx = (dxe.float() + dl @ b["router"]).bfloat16()
        return block.norm_backward(self.pre, dx, self.h0, self.norms[0], dh_add=dh)

    def update(self, step, lr):
        optim.step(self.plan, lr=lr, step=step, seed=step)
        if self.matrices is not None:
            muon.step(self.matrices, lr=lr)

    def check(self):
        """Raise on an error found on the device."""
        for b in self.bufs:
            layer.check(b)
        for b in self.balances:
            balance.check(b)
        if self.matrices is not None:
            muon.check(self.matrices)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--bits", type=int, choices=(32, 8), default=32, help="of the optimiser's states")
    ap.add_argument("--score", choices=("softmax", "sigmoid"), default="softmax")
    ap.add_argument("--optimizer", choices=("adamw", "muon"), default="adamw", help="of the matrices")
    ap.add_argument("--prec", choices=("bf16", "mxfp8", "mxfp8-w4", "fp8-block"), default="bf16", help="of the experts' products")
    a = ap.parse_args()
    T, d, f, E, k = 2048, 512, 256, 16, 2
    model = Stack(T, d, f, E, k, score=a.score, sequences=4, bits=a.bits, prec=a.prec, optimizer=a.optimizer)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    mix = torch.randn(d, d, generator=g, device="cuda") / math.sqrt(d)
    target = torch.tanh(h.float() @ mix)                       # synthetic: a map the blocks have to learn
    offsets = torch.tensor([0, 300, 1100, 1101, T], dtype=torch.int32, device="cuda")
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[1000:1100] = 0                                        # padding: no part in the losses
    kept = mask.float()[:, None]
    n = kept.sum() * d
    for t in range(1, a.steps + 1):
        x = model.forward(h, offsets, mask)
        off = (x.float() - target) * kept
        model.backward((2 * off / n).bfloat16())
        model.update(t, lr=3e-3)
        if t == 1 or t % 5 == 0 or t == a.steps:
            aux = sum(b.losses for b in model.balances).tolist()
            print(f"step {t:4d}  loss {float(off.square().sum() / n):.4f}  balance {aux[0]:.5f}  z {aux[1]:.5f}")
    model.check()


if __name__ == "__main__":
    main()
