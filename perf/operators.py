"""Cases of the operators around the MoE layer's training step, their plain forms and their definitions.

Three operators: the block norms (the norm before a block; the merge after it: the norm of the block's
output, its gate, the scaled residual and the next block's norm), the router's balance loss with its
per-expert counts, and the AdamW step over a list of tensors with 32-bit or 8-bit states.

``run`` computes a case in its plain form (torch operations in 32 bits) or, where ``own`` is true,
through the framework's entry points; ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

BLOCK = 128                      # elements that share a scale in the 8-bit states
BF16, F32 = "bf16", "fp32"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
SIZE = {BF16: 2, F32: 4}
EPS_NORM = 1e-6
ALPHA, BETA = 1.0, 0.5           # the merge's residual and branch scales
COEF, Z_COEF = 1e-2, 1e-3        # balance and z-loss coefficients
LR, BETA1, BETA2, EPS = 3e-4, 0.9, 0.95, 1e-8


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a DeepSeek-V3-width block while serving: latency only
        {"name": "merge token", "op": "merge_fwd", "T": 1, "d": 7168, "stream": BF16, "gate": "channel", "post": True,
         "next": True},
        # a ragged micro-batch with an fp32 residual stream and a sigmoid gate a token
        {"name": "merge ragged", "op": "merge_fwd", "T": 1237, "d": 2048, "stream": F32, "gate": "token", "post": True,
         "next": True},
        # the training step's batch at the DeepSeek-V3 width
        {"name": "merge batch", "op": "merge_fwd", "T": 16384, "d": 7168, "stream": BF16, "gate": "channel", "post": True,
         "next": True},
        {"name": "merge batch grads", "op": "merge_bwd", "T": 16384, "d": 7168, "stream": BF16, "gate": "channel",
         "post": True, "next": True},
        # the norm before the first block: its gradient joins the residual's, fp32 stream, the Mixtral width
        {"name": "norm grads", "op": "norm_bwd", "T": 8192, "d": 4096, "stream": F32},
        # the smallest router: a few hundred tokens, 8 experts
        {"name": "balance small", "op": "balance_fwd", "T": 256, "E": 8, "k": 2, "score": "softmax", "seqs": 1, "mask": False},
        # the DeepSeek-V3-shaped router: sigmoid scores, ragged sequences with padding
        {"name": "balance batch", "op": "balance_fwd", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "seqs": 9,
         "mask": True},
        {"name": "balance batch grads", "op": "balance_bwd", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "seqs": 9,
         "mask": True},
        # a long accumulation window over 128 experts: logits larger than the L2 cache
        {"name": "balance long grads", "op": "balance_bwd", "T": 393216, "E": 128, "k": 8, "score": "softmax", "seqs": 64,
         "mask": False},
        # many small tensors of odd sizes: norm weights, routers, small experts; fp32 gradients, no 16-bit copy
        {"name": "adamw many", "op": "adamw", "bits": 32, "grad": F32, "copy": False, "layers": 19, "E": 4, "d": 217,
         "f": 45},
        # one Qwen3-30B-A3B-shaped layer: fp32 master weights, bf16 gradients and the layer's bf16 copy
        {"name": "adamw layer", "op": "adamw", "bits": 32, "grad": BF16, "copy": True, "layers": 1, "E": 128, "d": 2048,
         "f": 768},
        {"name": "adamw layer 8-bit", "op": "adamw", "bits": 8, "grad": BF16, "copy": True, "layers": 1, "E": 128, "d": 2048,
         "f": 768},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["merge_fwd", "merge_bwd", "norm_fwd", "norm_bwd", "balance_fwd", "balance_bwd", "adamw", "adamw"])
    if op == "adamw":
        while True:
            c = {"op": op, "bits": rng.choice([8, 32]), "grad": rng.choice([BF16, F32]), "copy": rng.random() < 0.7,
                 "layers": _log_int(rng, 1, 40), "E": _log_int(rng, 1, 64), "d": 2 * _log_int(rng, 8, 1024) + 1,
                 "f": 2 * _log_int(rng, 8, 512) + 1}
            if sum(_sizes(c)) <= 200_000_000:
                return c
    if op.startswith("balance"):
        while True:
            E = rng.choice([8, 16, 60, 64, 128, 160, 256, 512, 2 * _log_int(rng, 2, 200) + 1])
            T = _log_int(rng, 1, 400_000) | 1
            if T * E <= 393216 * 128:
                break
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, E)), "score": rng.choice(["softmax", "sigmoid"]),
                "seqs": rng.choice([1, 1, _log_int(rng, 2, 100)]), "mask": rng.random() < 0.5}
    while True:
        T = _log_int(rng, 1, 30_000) | 1
        d = rng.choice([128, 1024, 2048, 4096, 7168, 8 * (2 * _log_int(rng, 4, 500) + 1)])
        if T * d <= 16384 * 7168:
            break
    c = {"op": op, "T": T, "d": d, "stream": rng.choice([BF16, F32])}
    if op.startswith("merge"):
        c.update(gate=rng.choice(["none", "channel", "token"]), post=rng.random() < 0.8, next=rng.random() < 0.8)
        if c["stream"] == F32 and T * d > 16384 * 4096:
            c["stream"] = BF16
    return c


def _sizes(c):
    """Elements of the tensors of `layers` MoE layers: gate/up and down experts, router, two norm weights."""
    E, d, f = c["E"], c["d"], c["f"]
    return [E * 2 * f * d, E * d * f, E * d, d, d] * c["layers"]


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        state = 2 * (4 + 4) if case["bits"] == 32 else 2 * (1 + 1) + 2 * 2 * 4 / BLOCK + (1 + 1 + 2 + 2) + 8 / BLOCK
        # 8-bit states come back as the values they stand for: read once more, written as bf16
        return {"bytes": n * (8 + state + SIZE[case["grad"]] + (2 if case["copy"] else 0)), "flops": 14.0 * n}
    if op.startswith("balance"):
        n = case["T"] * case["E"]
        if op == "balance_fwd":
            return {"bytes": 4.0 * n + 4.0 * case["T"] * case["k"] + 8.0 * case["seqs"] * case["E"], "flops": 6.0 * n}
        return {"bytes": 12.0 * n + 4.0 * case["seqs"] * case["E"], "flops": 10.0 * n}
    n, s = case["T"] * case["d"], SIZE[case["stream"]]
    if op == "norm_fwd":
        return {"bytes": n * (s + 2.0), "flops": 4.0 * n}
    if op == "norm_bwd":
        return {"bytes": n * (2.0 + 3 * s), "flops": 10.0 * n}
    nx = 2 if case["next"] else 0
    if op == "merge_fwd":
        return {"bytes": n * (2.0 * s + 2 + nx), "flops": 12.0 * n}
    need_h, need_y = case["next"], case["post"] or case["gate"] != "none"
    return {"bytes": n * (2.0 * s + 2 + nx + (s if need_h else 0) + (2 if need_y else 0)), "flops": 24.0 * n}


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["op"].split("_")[0]
    return {"merge": _prepare_norm, "norm": _prepare_norm, "balance": _prepare_balance, "adamw": _prepare_adamw}[kind](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_norm(case, g):
    T, d, st = case["T"], case["d"], DTYPE[case["stream"]]
    s = {"case": case}
    h = _randn(g, T, d) * 2.0
    h[:, :: max(1, d // 5)] *= 20.0                      # a few channels of the stream carry large values
    s["h"] = h.to(st)
    merge = case["op"].startswith("merge")
    s["w"] = 1.0 + 0.1 * _randn(g, d) if not merge or case["next"] else None
    if merge:
        s["y"] = (_randn(g, T, d) * 0.3).bfloat16()
        s["w_post"] = 0.5 + 0.1 * _randn(g, d) if case["post"] else None
        s["gate"] = {"none": None, "channel": 0.3 + 0.1 * _randn(g, d), "token": _randn(g, T)}[case["gate"]]
    if case["op"].endswith("bwd"):
        s["dh"] = (_randn(g, T, d) * 1e-3).to(st)
        s["dx"] = (_randn(g, T, d) * 1e-2).bfloat16() if s["w"] is not None else None
    if own:
        from dropless_mixture_experts_warp_gb300 import block
        gate = case.get("gate", "none")
        s["b"] = block.allocate(block.dims_of(T, d, stream=case["stream"], weights="fp32", gate=gate,
                                              gate_act="sigmoid" if gate == "token" else "identity", eps=EPS_NORM,
                                              alpha=ALPHA, beta=BETA))
    return s


def _prepare_balance(case, g):
    T, E, S = case["T"], case["E"], case["seqs"]
    logits = _randn(g, T, E) + 0.7 * _randn(g, E)        # some experts are more popular than others
    s = {"case": case, "logits": logits, "idx": torch.topk(logits, case["k"], dim=1).indices.int()}
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")).values
    if S > 4:
        cuts[2] = cuts[1]                                # one sequence is empty
    zero = torch.zeros(1, dtype=cuts.dtype, device="cuda")
    s["offsets"] = torch.cat([zero, cuts, zero + T]).int()
    pos = torch.arange(T, device="cuda")
    s["seq"] = (torch.searchsorted(s["offsets"].long(), pos, right=True) - 1).clamp_(0, S - 1)
    s["mask"] = None
    if case["mask"]:                                     # every sequence ends in padding; one is padding alone
        start, end = s["offsets"].long()[:-1], s["offsets"].long()[1:]
        keep = (end - start).float() * (0.5 + 0.5 * torch.rand(S, generator=g, device="cuda"))
        if S > 4:
            keep[S - 1] = 0.0
        s["mask"] = ((pos - start[s["seq"]]) < keep.ceil()[s["seq"]]).to(torch.uint8)
    if case["op"] == "balance_bwd":                      # what the forward left, and the router's own gradient
        member = torch.nn.functional.one_hot(s["seq"], S).t().float()
        if s["mask"] is not None:
            member = member * s["mask"]
        hits = torch.zeros(T, E, device="cuda").scatter_(1, s["idx"].long(), 1.0)
        s["counts"], s["tokens"] = (member @ hits).round().int(), member.sum(1).int()
        s["d_logits"] = _randn(g, T, E) * (0.02 / (T * E))
        s["grad"] = torch.tensor([1.0, 0.5], device="cuda")
    if own:
        from dropless_mixture_experts_warp_gb300 import balance
        s["o"] = balance.allocate(T, E, case["k"], score=case["score"], sequences=S)
        if "counts" in s:
            s["o"].counts.copy_(s["counts"])
            s["o"].seq_tokens.copy_(s["tokens"])
    return s


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    starts, at = [], 0
    for n in sizes:                                      # the tensors are views of flat buffers, 128-element aligned
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    big = lambda dt: torch.zeros(at, dtype=dt, device="cuda")  # noqa: E731
    views = lambda flat: [flat[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
    s = {"case": case, "step": 10, "starts": starts, "sizes": sizes, "w": big(torch.float32), "g": big(DTYPE[case["grad"]]),
         "copy": big(torch.bfloat16) if case["copy"] else None,
         "decay": [0.1 if i % 5 < 3 else 0.0 for i in range(len(sizes))]}   # matrices decay, norm weights do not
    eight = case["bits"] == 8
    s["m"], s["v"] = (big(torch.int8), big(torch.uint8)) if eight else (big(torch.float32), big(torch.float32))
    if eight:
        s["ms"], s["vs"] = (torch.zeros(at // BLOCK, device="cuda") for _ in range(2))
    # the tensor and the first element of every block
    counts = torch.tensor([-(-n // BLOCK) for n in sizes], device="cuda")
    s["tensor"] = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), counts)
    s["first"] = torch.arange(at // BLOCK, device="cuda") * BLOCK - torch.tensor(starts, device="cuda")[s["tensor"]]
    s["wd"] = torch.tensor(s["decay"], device="cuda")[s["tensor"]][:, None]
    left = torch.tensor(sizes, device="cuda")[s["tensor"]] - s["first"]
    inside = (torch.arange(BLOCK, device="cuda")[None, :] < left[:, None]).view(-1)
    s["w"].normal_(generator=g).mul_(0.02).mul_(inside)
    rough = torch.empty(at, device="cuda")
    s["g"].copy_(rough.normal_(generator=g).mul_(1e-3).mul_(inside))
    rough.normal_(generator=g).mul_(3e-4).mul_(inside)                     # the first moment
    if eight:
        b = rough.view(-1, BLOCK)
        s["ms"].copy_(b.abs().amax(1))
        s["m"].view(-1, BLOCK).copy_(b.sign() * (127 * (b.abs() / s["ms"].clamp_min(1e-30)[:, None]).sqrt()).round())
    else:
        s["m"].copy_(rough)
    rough.normal_(generator=g).mul_(1e-3).square_().add_(1e-8).mul_(inside)  # the second
    if eight:
        b = rough.view(-1, BLOCK)
        s["vs"].copy_(b.amax(1))
        s["v"].view(-1, BLOCK).copy_((255 * (b / s["vs"].clamp_min(1e-30)[:, None]).sqrt().sqrt()).round())
        s["mv"], s["vv"] = big(torch.bfloat16), big(torch.bfloat16)
    else:
        s["v"].copy_(rough)
    if own:
        from dropless_mixture_experts_warp_gb300 import optim
        s["plan"] = optim.plan(views(s["w"]), views(s["g"]), copies=views(s["copy"]) if case["copy"] else None,
                               bits=case["bits"], weight_decay=s["decay"], m=views(s["m"]), v=views(s["v"]),
                               m_scale=_scales(s, "ms") if eight else None, v_scale=_scales(s, "vs") if eight else None)
        if eight:
            s["out"] = views(s["mv"]), views(s["vv"])
    return s


def _scales(s, key):
    return [s[key][a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(s["starts"], s["sizes"])]


# ------------------------------------------------------------------------------------ one pass

def run(state):
    return {"merge_fwd": _merge_fwd, "merge_bwd": _merge_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd,
            "balance_fwd": _balance_fwd, "balance_bwd": _balance_bwd, "adamw": _adamw}[state["case"]["op"]](state)


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS_NORM)


def _act(s):
    """The gate as a factor of [T, d] values, and its derivative by the gate's input."""
    kind = s["case"]["gate"]
    if kind == "none":
        return 1.0, None
    if kind == "channel":
        return s["gate"][None, :], 1.0
    a = torch.sigmoid(s["gate"])[:, None]
    return a, a * (1 - a)


def _norm_fwd(s):
    if own:
        from dropless_mixture_experts_warp_gb300 import block
        return block.norm_forward(s["b"], s["h"], s["w"])
    h = s["h"].float()
    return (h * _rms(h) * s["w"]).bfloat16()


def _norm_bwd(s):
    if own:
        from dropless_mixture_experts_warp_gb300 import block
        b = s["b"]
        block.norm_backward(b, s["dx"], s["h"], s["w"], dh_add=s["dh"])
        return {"dh": b.dh, "dw": b.dw}
    h, dx = s["h"].float(), s["dx"].float()
    r = _rms(h)
    hh, n = h * r, dx * s["w"]
    dh = s["dh"].float() + r * (n - hh * (n * hh).mean(-1, keepdim=True))
    return {"dh": dh.to(s["h"].dtype), "dw": (dx * hh).double().sum(0).float()}


def _merge_fwd(s):
    if own:
        from dropless_mixture_experts_warp_gb300 import block
        b = s["b"]
        block.merge_forward(b, s["h"], s["y"], w_post=s["w_post"], gate=s["gate"], w_next=s["w"])
        return {"h": b.h_out, "x": b.x if s["w"] is not None else None}
    z = s["y"].float()
    if s["w_post"] is not None:
        z = z * _rms(z) * s["w_post"]
    h = ALPHA * s["h"].float() + BETA * _act(s)[0] * z
    x = (h * _rms(h) * s["w"]).bfloat16() if s["w"] is not None else None
    return {"h": h.to(s["h"].dtype), "x": x}


def _merge_bwd(s):
    """Here s["h"] is the stream that the forward wrote."""
    gate = s["case"]["gate"]
    if own:
        from dropless_mixture_experts_warp_gb300 import block
        b = s["b"]
        block.merge_backward(b, s["dh"], s["dx"], s["h"], s["y"], w_post=s["w_post"], gate=s["gate"], w_next=s["w"])
        return {"dh": b.dh, "dy": b.dy, "dw_post": b.dw_post if s["w_post"] is not None else None,
                "dgate": b.dgate if gate != "none" else None, "dw_next": b.dw if s["w"] is not None else None}
    h, y, D = s["h"].float(), s["y"].float(), s["dh"].float()
    dw_next = dw_post = dgate = None
    if s["w"] is not None:
        r, dx = _rms(h), s["dx"].float()
        hh, n = h * r, dx * s["w"]
        D = D + r * (n - hh * (n * hh).mean(-1, keepdim=True))
        dw_next = (dx * hh).double().sum(0).float()
    a, da = _act(s)
    dz = BETA * a * D
    z = y
    if s["w_post"] is not None:
        r = _rms(y)
        yh = y * r
        z, q = yh * s["w_post"], dz * s["w_post"]
        dw_post = (dz * yh).double().sum(0).float()
        dy = r * (q - yh * (q * yh).mean(-1, keepdim=True))
    else:
        dy = dz
    if gate == "channel":
        dgate = (BETA * D * z).double().sum(0).float()
    elif gate == "token":
        dgate = ((BETA * D * z).double().sum(1) * da[:, 0]).float()
    return {"dh": (ALPHA * D).to(s["h"].dtype), "dy": dy.bfloat16(), "dw_post": dw_post, "dgate": dgate, "dw_next": dw_next}


def _probabilities(l, score):
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
    else:
        e = torch.sigmoid(l)
    return e / e.sum(1, keepdim=True)


def _lse(l):
    top = l.amax(1)
    return top + torch.log(torch.exp(l - top[:, None]).sum(1))


def _members(s):
    """[sequences, tokens]: 1 where the token counts in the sequence."""
    m = (s["seq"][None, :] == torch.arange(s["case"]["seqs"], device="cuda")[:, None]).double()
    return m if s["mask"] is None else m * s["mask"]


def _balance_fwd(s):
    c = s["case"]
    if own:
        from dropless_mixture_experts_warp_gb300 import balance
        o = s["o"]
        balance.forward(o, s["logits"], s["idx"], seq_offsets=s["offsets"], mask=s["mask"], coef=COEF, z_coef=Z_COEF)
        return {"losses": o.losses, "counts": o.counts, "prob_mean": o.prob_mean, "tokens": o.seq_tokens}
    member = _members(s)
    tokens = member.sum(1)
    hits = torch.zeros_like(s["logits"]).scatter_(1, s["idx"].long(), 1.0)
    counts = member @ hits.double()
    mean = (member @ _probabilities(s["logits"], c["score"]).double()) / tokens.clamp_min(1)[:, None]
    f = counts * c["E"] / (c["k"] * tokens.clamp_min(1)[:, None])
    balance_loss = (f * mean).sum() / (tokens > 0).sum().clamp_min(1)
    z_loss = (member.sum(0) * _lse(s["logits"]).double().square()).sum() / tokens.sum().clamp_min(1)
    return {"losses": torch.stack([COEF * balance_loss, Z_COEF * z_loss]).float(), "counts": counts.round().int(),
            "prob_mean": mean.float(), "tokens": tokens.int()}


def _balance_bwd(s):
    c, l = s["case"], s["logits"]
    if own:
        from dropless_mixture_experts_warp_gb300 import balance
        balance.backward(s["o"], l, s["d_logits"], seq_offsets=s["offsets"], mask=s["mask"], coef=COEF, z_coef=Z_COEF,
                         grad=s["grad"])
        return s["d_logits"]
    n = s["tokens"].clamp_min(1).float()
    f = s["counts"] * (c["E"] / c["k"]) / n[:, None]
    per_seq = COEF / ((s["tokens"] > 0).sum().clamp_min(1) * n)
    keep = torch.ones_like(l[:, 0]) if s["mask"] is None else s["mask"].float()
    p, ft = _probabilities(l, c["score"]), f[s["seq"]]
    d = (s["grad"][0] * per_seq[s["seq"]] * keep)[:, None] * p * (ft - (ft * p).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d * torch.sigmoid(-l)
    scale = s["grad"][1] * (2 * Z_COEF) / s["tokens"].sum().clamp_min(1)
    d = d + (scale * keep * _lse(l))[:, None] * _probabilities(l, "softmax")
    s["d_logits"] += d
    return s["d_logits"]


LOW = 0xFFFFFFFF


def _mix(x):
    """A 32-bit mixing function, on non-negative 64-bit values."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & LOW
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & LOW
    return x ^ (x >> 16)


def _random(s, seed):
    """The two 16-bit random numbers of every element: from the seed, the step, the tensor and the element."""
    base = _mix((_mix(torch.tensor(seed, device="cuda")) + s["step"]) & LOW)
    at = s["first"][:, None] + torch.arange(BLOCK, device="cuda")[None, :]
    key = _mix((base + s["tensor"][:, None] * 0x6A09E667 + (at >> 32) * 0xBB67AE85) & LOW)
    x = _mix(((at & LOW) * 0x9E3779B9 + key) & LOW)
    return x & 0xFFFF, x >> 16


def _adamw(s):
    c = s["case"]
    s["step"] += 1
    if own:
        from dropless_mixture_experts_warp_gb300 import optim
        optim.step(s["plan"], lr=LR, step=s["step"], beta1=BETA1, beta2=BETA2, eps=EPS, seed=7)
        if c["bits"] == 8:
            optim.values(s["plan"], *s["out"])
    else:
        g, w = s["g"].float().view(-1, BLOCK), s["w"].view(-1, BLOCK)
        if c["bits"] == 8:
            k, q = s["m"].view(-1, BLOCK).float(), s["v"].view(-1, BLOCK).float()
            m = s["ms"][:, None] * (k * k.abs() * (1.0 / 16129))
            v = s["vs"][:, None] * (q * q * (1.0 / 65025)).square()
        else:
            m, v = s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK)
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + (g * g) * (1 - BETA2)
        update = (m * (1 / (1 - BETA1 ** s["step"]))) / ((v * (1 / (1 - BETA2 ** s["step"]))).sqrt() + EPS)
        w.copy_(w - LR * (update + s["wd"] * w))
        if s["copy"] is not None:
            s["copy"].copy_(s["w"])
        if c["bits"] == 8:
            _store8(s, m, v)
        else:
            s["m"].copy_(m.view(-1))
            s["v"].copy_(v.view(-1))
    out = {"w": s["w"], "copy": s["copy"]}
    out.update({"m": s["mv"], "v": s["vv"]} if c["bits"] == 8 else {"m": s["m"], "v": s["v"]})
    return out


def _store8(s, m, v):
    """Codes of the moments, rounded at random between neighbours so that a code's mean is the value; in 64
    bits, for values next to a border."""
    low, high = _random(s, 7)
    tiny = torch.finfo(torch.float32).tiny
    ms, vs = m.abs().amax(1), v.amax(1)
    ms, vs = torch.where(ms < tiny, 0.0, ms), torch.where(vs < tiny, 0.0, vs)
    x = m.abs().double() / torch.where(ms > 0, ms, 1.0)[:, None] * 16129 * (ms > 0)[:, None]
    k = x.sqrt().floor()
    k = k + ((low + 0.5) / 65536 * (2 * k + 1) < x - k * k)
    s["m"].view(-1, BLOCK).copy_(m.sign() * k.clamp_max(127))
    x = v.double() / torch.where(vs > 0, vs, 1.0)[:, None] * 255.0 ** 4 * (vs > 0)[:, None]
    k = x.sqrt().sqrt().floor()
    k = k + ((high + 0.5) / 65536 * ((k + 1) ** 4 - k ** 4) < x - k ** 4)
    s["v"].view(-1, BLOCK).copy_(torch.where(x > 0, k.clamp(1, 255), 0.0))
    s["ms"].copy_(ms)
    s["vs"].copy_(vs)
    k, q = s["m"].view(-1, BLOCK).float(), s["v"].view(-1, BLOCK).float()
    s["mv"].view(-1, BLOCK).copy_(ms[:, None] * (k * k.abs() * (1.0 / 16129)))
    s["vv"].view(-1, BLOCK).copy_(vs[:, None] * (q * q * (1.0 / 65025)).square())


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(s)
    if op.startswith("balance"):
        return _exact_balance(s)
    return _exact_norm(s)


def _exact_norm(s):
    """The forward's formula in 64 bits; gradients by automatic differentiation of it."""
    case = s["case"]
    leaf = lambda t: None if t is None else t.double().requires_grad_(case["op"].endswith("bwd"))  # noqa: E731
    norm = lambda t, w: t / (t.pow(2).mean(1, keepdim=True) + EPS_NORM).sqrt() * w  # noqa: E731
    h, w = leaf(s["h"]), leaf(s["w"])
    if case["op"] == "norm_fwd":
        return norm(h, w)
    if case["op"] == "norm_bwd":
        dh, dw = torch.autograd.grad(norm(h, w), [h, w], s["dx"].double())
        return {"dh": dh + s["dh"].double(), "dw": dw}
    y, w_post, gate = leaf(s["y"]), leaf(s["w_post"]), leaf(s["gate"])
    z = y if w_post is None else norm(y, w_post)
    if case["gate"] == "channel":
        z = z * gate
    elif case["gate"] == "token":
        z = z / (1 + torch.exp(-gate))[:, None]
    if case["op"] == "merge_fwd":
        out = ALPHA * h + BETA * z
        return {"h": out, "x": None if w is None else norm(out, w)}
    # the stream after the merge is an input of the backward: differentiate the two halves on either side of it
    D = s["dh"].double()
    dw_next = None
    if w is not None:
        more, dw_next = torch.autograd.grad(norm(h, w), [h, w], s["dx"].double())
        D = D + more
    wanted = [t for t in (y, w_post, gate) if t is not None]
    grads = dict(zip(map(id, wanted), torch.autograd.grad(BETA * z, wanted, D)))
    return {"dh": ALPHA * D, "dy": grads[id(y)], "dw_post": grads.get(id(w_post)), "dgate": grads.get(id(gate)),
            "dw_next": dw_next}


def _exact_balance(s):
    """Sequence by sequence; gradients by automatic differentiation of the losses."""
    c = s["case"]
    bwd = c["op"] == "balance_bwd"
    l = s["logits"].double().requires_grad_(bwd)
    ends = s["offsets"].tolist()
    kept = [torch.arange(a, b, device="cuda") for a, b in zip(ends, ends[1:])]
    if s["mask"] is not None:
        kept = [k[s["mask"][k] != 0] for k in kept]
    counts = torch.stack([torch.bincount(s["idx"][k].reshape(-1).long(), minlength=c["E"]) for k in kept])
    full = max(1, sum(len(k) > 0 for k in kept))
    means, loss = [], 0.0
    for k, n in zip(kept, counts):
        if c["score"] == "softmax":
            p = torch.softmax(l[k], 1)
        else:
            p = 1 / (1 + torch.exp(-l[k]))
            p = p / p.sum(1, keepdim=True)
        means.append(p.sum(0) / max(1, len(k)))
        loss = loss + (n.double() * means[-1]).sum() * c["E"] / (c["k"] * max(1, len(k))) / full
    every = torch.cat(kept)
    z = (torch.logsumexp(l[every], 1) ** 2).sum() / max(1, len(every))
    if not bwd:
        return {"losses": torch.stack([COEF * loss, Z_COEF * z]), "counts": None, "prob_mean": torch.stack(means),
                "tokens": None}
    total = s["grad"][0].double() * COEF * loss + s["grad"][1].double() * Z_COEF * z
    return s["d_logits"].double() + torch.autograd.grad(total, l)[0]


def _exact_adamw(s):
    c = s["case"]
    t = s["step"] + 1
    g, w, m, v = (s[key].view(-1, BLOCK).double() for key in ("g", "w", "m", "v"))
    if c["bits"] == 8:
        m = s["ms"].double()[:, None] * m.sign() * (m / 127) ** 2
        v = s["vs"].double()[:, None] * (v / 255) ** 4
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g ** 2 - v)
    rate = LR / (1 - BETA1 ** t)
    w = w * (1 - LR * s["wd"].double()) - rate * m / (EPS + torch.sqrt(v / (1 - BETA2 ** t)))
    if c["bits"] == 8:
        low, high = _random({**s, "step": t}, 7)
        m, v = _nearby(m, low, 127, 2), _nearby(v, high, 255, 4)
    w = w.view(-1)
    return {"w": w, "copy": w if c["copy"] else None, "m": m.view(-1), "v": v.view(-1)}


def _nearby(x, random, top, power):
    """x as largest * (code / top) ** power, the code one of the two around it: the upper one with the chance that
    makes the mean x; no value but zero becomes zero in an unsigned state."""
    largest = x.abs().amax(1, keepdim=True)
    share = torch.where(largest > 0, x.abs() / largest.clamp_min(1e-300), 0.0)
    code = torch.floor(share ** (1.0 / power) * top + 1e-12)
    under, over = (code / top) ** power, ((code + 1) / top) ** power
    code = torch.where((share - under) / (over - under) > (random + 0.5) / 65536, code + 1, code).clamp_max(top)
    if power == 4:
        code = torch.where(share > 0, code.clamp_min(1), code)
    return x.sign() * largest * (code / top) ** power
