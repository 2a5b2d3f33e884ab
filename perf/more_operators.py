"""Cases of the 8-bit products with a scale for each block of 128 and of the orthogonalised update.

Five operators: the quantiser of activations (blocks of 128 along rows and, for weight gradients, down columns), the
product of quantised rows with quantised weights (one matrix, or one for each expert), the ragged weight gradient, the
layer's forward through them, and the update orthogonalised by Newton-Schulz products (Muon).

``run`` computes a case in its plain form (torch operations in 32 bits) or, where ``own`` is true, through the
framework's entry points; ``exact`` computes it in 64 bits from the definition.
"""
import math
import random

import torch

own = False

BLOCK = 128
TOP = 448.0                                  # the largest E4M3 value
FLOOR = 2.0 ** -64                           # a block's largest value counts as at least this
E4M3 = torch.float8_e4m3fn
MOMENTUM, DECAY, RMS = 0.95, 0.1, 0.2
LR = 2e-4
STEPS = [(3.4445, -4.7750, 2.0315)] * 5      # a, b, c of each Newton-Schulz step


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # eight tokens of a serving step before a product at the DeepSeek-V3 width: latency only
        {"name": "quantize tokens", "op": "quantize", "R": 8, "C": 7168, "both": False},
        # a training batch at that width, for the forward product and the weight gradient
        {"name": "quantize batch", "op": "quantize", "R": 16384, "C": 7168, "both": True},
        # a shared expert's gate/up product for a few tokens: bound by reading the weights
        {"name": "product tokens", "op": "product", "E": 1, "R": 5, "N": 4096, "K": 7168, "skew": 0.0, "wide": False},
        # an output projection of odd sizes, its input gradient (the weights read along the other axis)
        {"name": "product odd", "op": "product", "E": 1, "R": 1237, "N": 2064, "K": 1456, "skew": 0.0, "wide": True},
        # 64 tokens of a serving step over 256 experts, gate/up: a few rows an expert, all weights read
        {"name": "product experts decode", "op": "product", "E": 256, "R": 512, "N": 4096, "K": 7168, "skew": 0.6,
         "wide": False},
        # a training batch over 32 experts with a skewed router, gate/up
        {"name": "product experts batch", "op": "product", "E": 32, "R": 32768, "N": 4096, "K": 7168, "skew": 0.8,
         "wide": False},
        # one Qwen3-30B-A3B-shaped expert's down weights, one expert's rows
        {"name": "weight grad one", "op": "wgrad", "E": 1, "R": 900, "N": 2048, "K": 768, "skew": 0.0},
        {"name": "weight grad batch", "op": "wgrad", "E": 32, "R": 32768, "N": 7168, "K": 2048, "skew": 0.8},
        # four tokens through a DeepSeek-V3-shaped layer: routing, dispatch, both products, combine
        {"name": "layer tokens", "op": "layer", "T": 4, "d": 7168, "f": 2048, "E": 256, "k": 8, "score": "sigmoid"},
        # a prompt batch through a Qwen3-30B-A3B-shaped layer
        {"name": "layer batch", "op": "layer", "T": 16384, "d": 2048, "f": 768, "E": 128, "k": 8, "score": "softmax"},
        # a router's and small experts' matrices of odd sizes: launches and latency
        {"name": "muon small", "op": "orthogonalize", "B": 6, "m": 131, "n": 72, "grad": "bf16"},
        # the gate, up and down matrices of 16 Qwen3-235B-A22B-shaped experts in one optimiser step
        {"name": "muon experts", "op": "muon", "E": 16, "d": 4096, "f": 1536, "grad": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "wgrad", "layer", "orthogonalize", "muon"])
    if op == "quantize":
        while True:
            c = {"op": op, "R": _log_int(rng, 1, 30_000) | 1, "C": 16 * _log_int(rng, 4, 512), "both": rng.random() < 0.5}
            if c["R"] * c["C"] <= 16384 * 7168:
                return c
    if op in ("product", "wgrad"):
        while True:
            E = rng.choice([1, 1, 8, 16, 60, 128, 256])
            c = {"op": op, "E": E, "R": _log_int(rng, 1 if op == "product" else 64, 40_000),
                 "N": 16 * _log_int(rng, 8, 512), "K": 16 * _log_int(rng, 8, 512), "skew": round(rng.uniform(0.0, 1.0), 2)}
            if op == "product":
                c["wide"] = rng.random() < 0.4
            if c["R"] * c["N"] * c["K"] <= 8192 * 4096 * 7168 and E * c["N"] * c["K"] <= 1 << 31:
                return c
    if op == "layer":
        while True:
            E = rng.choice([8, 16, 60, 128, 256])
            c = {"op": op, "T": _log_int(rng, 1, 16_000), "d": 128 * _log_int(rng, 2, 56), "f": 128 * _log_int(rng, 1, 24),
                 "E": E, "k": rng.randint(1, min(8, E)), "score": rng.choice(["softmax", "sigmoid"])}
            if E * c["d"] * c["f"] <= 1 << 30 and c["T"] * c["k"] * c["d"] * c["f"] <= 1 << 37:
                return c
    if op == "orthogonalize":
        while True:
            c = {"op": op, "B": _log_int(rng, 1, 40), "m": _log_int(rng, 16, 4000), "n": _log_int(rng, 16, 4000),
                 "grad": rng.choice(["bf16", "fp32"])}
            if c["B"] * c["m"] * c["n"] * min(c["m"], c["n"]) <= 1 << 36:
                return c
    while True:
        c = {"op": op, "E": _log_int(rng, 1, 40), "d": _log_int(rng, 32, 4000), "f": _log_int(rng, 32, 2000),
             "grad": rng.choice(["bf16", "fp32"])}
        if c["E"] * c["d"] * c["f"] * min(c["d"], c["f"]) <= 1 << 35:
            return c


def _shapes(c):
    """The matrices of a muon case: gate and up of every expert, down of every expert."""
    return [(2 * c["E"], c["f"], c["d"]), (c["E"], c["d"], c["f"])]


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["R"] * case["C"]
        return {"bytes": n * (4.0 if case["both"] else 3.0) + 4.0 * n / BLOCK * (2 if case["both"] else 1), "flops": 3.0 * n}
    if op in ("product", "wgrad"):
        E, R, N, K = (case[x] for x in ("E", "R", "N", "K"))
        used = min(E, R)                                           # experts that have rows, at most
        if op == "product":
            return {"bytes": 1.0 * R * K + 1.0 * used * N * K + 2.0 * R * N, "flops": 2.0 * R * N * K}
        return {"bytes": 1.0 * R * (N + K) + 2.0 * E * N * K, "flops": 2.0 * R * N * K}
    if op == "layer":
        T, d, f, E, k = (case[x] for x in ("T", "d", "f", "E", "k"))
        used = min(E, T * k)
        return {"bytes": 3.0 * used * d * f + 4.0 * T * d + 4.0 * T * E, "flops": 6.0 * T * k * d * f}
    if op == "orthogonalize":
        shapes, moved = [(case["B"], case["m"], case["n"])], (2 if case["grad"] == "bf16" else 4) + 2
    else:
        shapes, moved = _shapes(case), (2 if case["grad"] == "bf16" else 4) + 16 + 2
    flops = sum(len(STEPS) * b * (3.0 * min(m, n) ** 2 * max(m, n) + 1.0 * min(m, n) ** 3) for b, m, n in shapes)
    return {"bytes": float(sum(b * m * n for b, m, n in shapes)) * moved, "flops": flops}


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = {"quantize": _prepare_quantize, "product": _prepare_product, "wgrad": _prepare_wgrad, "layer": _prepare_layer,
            "orthogonalize": _prepare_orthogonalize, "muon": _prepare_muon}
    return kind[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, R, C):
    """Rows of different sizes with a few large channels, as the inputs of an MLP have them."""
    x = _randn(g, R, C) * (0.5 + torch.rand(R, 1, generator=g, device="cuda"))
    x[:, 3:: max(4, C // 7)] *= 12.0
    return x.bfloat16()


def _prepare_quantize(case, g):
    s = {"case": case, "x": _activations(g, case["R"], case["C"])}
    if own:
        from dropless_mixture_experts_warp_gb300 import fp8
        s["rows"] = fp8.allocate_rows(case["R"], case["C"], both=case["both"])
    return s


def _segments(case):
    """Rows of each expert (a skewed router's, the same for every seed as they shape the buffers), and the offsets of
    their segments: multiples of 128."""
    E, R = case["E"], case["R"]
    if E == 1:
        return [R], [0, -(-R // BLOCK) * BLOCK]
    r = random.Random(E * 65537 + R)
    order = list(range(E))
    r.shuffle(order)
    share = [(order[e] + 1.0) ** -case["skew"] for e in range(E)]
    total = sum(share)
    counts = [int(R * p / total) for p in share]
    while sum(counts) < R:
        counts[r.randrange(E)] += 1
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + -(-n // BLOCK) * BLOCK)
    return counts, offsets


def _weights(g, E, N, K):
    """Codes and block scales as a checkpoint holds them."""
    codes = _randn(g, E, N, K).mul_(100.0).clamp_(-TOP, TOP).to(E4M3)
    scales = (0.5 + torch.rand(E, -(-N // BLOCK), -(-K // BLOCK), generator=g, device="cuda")) * (0.01 / math.sqrt(K))
    return codes, scales


def _rows_with_padding(g, case, counts, offsets, C):
    """Activations in the padded row space: zero rows behind each segment's own."""
    rows = case["R"] if case["E"] == 1 and case["op"] == "product" else offsets[-1]
    x = _activations(g, rows, C)
    if rows != case["R"]:
        at = torch.arange(rows, device="cuda")
        off = torch.tensor(offsets, device="cuda")
        e = torch.searchsorted(off, at, right=True) - 1
        keep = (at - off[e]) < torch.tensor(counts, device="cuda")[e.clamp(max=len(counts) - 1)]
        x = x * keep[:, None]
    return x


def _prepare_product(case, g):
    counts, offsets = _segments(case)
    wide = case["wide"]                                            # rows of N values times the weights: an input gradient
    x = _rows_with_padding(g, case, counts, offsets, case["N"] if wide else case["K"])
    codes, scales = _quantize_rows(x.float())
    w, ws = _weights(g, case["E"], case["N"], case["K"])
    out = torch.zeros(x.shape[0], case["K"] if wide else case["N"], dtype=torch.bfloat16, device="cuda")
    s = {"case": case, "codes": codes, "scales": scales, "w": w, "ws": ws, "offsets": None, "cap": max(counts),
         "segments": offsets, "out": out}
    if case["E"] > 1:
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    if wide:
        s["w_t"] = w.transpose(1, 2).contiguous()                  # as a training step keeps them beside the others
    if own:
        from dropless_mixture_experts_warp_gb300 import fp8
        s["a"] = fp8.rows_of(codes, scales)
        s["b"] = fp8.weights_of(w, ws, codes_t=s.get("w_t"))
    return s


def _prepare_wgrad(case, g):
    counts, offsets = _segments(case)
    dy = _rows_with_padding(g, case, counts, offsets, case["N"])
    x = _rows_with_padding(g, case, counts, offsets, case["K"])
    s = {"case": case, "cap": -(-max(counts) // BLOCK) * BLOCK, "segments": offsets,
         "out": torch.zeros(case["E"], case["N"], case["K"], dtype=torch.bfloat16, device="cuda"),
         "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda") if case["E"] > 1 else None}
    s["dy_t"], s["dy_s"] = _quantize_rows(dy.t().float())
    s["x_t"], s["x_s"] = _quantize_rows(x.t().float())
    if own:
        from dropless_mixture_experts_warp_gb300 import fp8
        s["dy"] = fp8.rows_of(codes_t=s["dy_t"], scales_t=s["dy_s"])
        s["x"] = fp8.rows_of(codes_t=s["x_t"], scales_t=s["x_s"])
    return s


def _prepare_layer(case, g):
    T, d, f, E, k = (case[x] for x in ("T", "d", "f", "E", "k"))
    logits = _randn(g, T, E) + 0.5 * _randn(g, E)
    top = torch.topk(logits, k, dim=1).indices
    s = {"case": case, "x": _randn(g, T, d).bfloat16(), "logits": logits,
         "cap": int(torch.bincount(top.reshape(-1), minlength=E).max())}
    s["wgu"], s["sgu"] = _weights(g, E, 2 * f, d)
    s["wd"], s["sd"] = _weights(g, E, d, f)
    if own:
        from dropless_mixture_experts_warp_gb300 import fp8, layer
        s["b"] = layer.allocate(layer.dims_of(T, d, f, E, k, score=case["score"], prec="fp8-block"), train=False)
        layer.use_weights(s["b"], fp8.weights_of(s["wgu"], s["sgu"]), fp8.weights_of(s["wd"], s["sd"]))
    return s


def _matrices(g, b, m, n, dtype):
    """Gradients: a few strong directions under noise."""
    r = max(1, min(m, n) // 16)
    x = torch.bmm(_randn(g, b, m, r), _randn(g, b, r, n)) * (2.0 / math.sqrt(r)) + _randn(g, b, m, n)
    return (x * 1e-4).to(dtype)


def _prepare_orthogonalize(case, g):
    x = _matrices(g, case["B"], case["m"], case["n"], torch.bfloat16 if case["grad"] == "bf16" else torch.float32)
    s = {"case": case, "x": x, "out": torch.empty_like(x, dtype=torch.bfloat16)}
    if own:
        from dropless_mixture_experts_warp_gb300 import muon
        s["plan"] = muon.workspace([x.shape])
    return s


def _prepare_muon(case, g):
    kind = torch.bfloat16 if case["grad"] == "bf16" else torch.float32
    s = {"case": case, "w": [], "m": [], "grads": []}
    for b, m, n in _shapes(case):
        s["w"].append(_randn(g, b, m, n) * 0.02)
        s["m"].append(_matrices(g, b, m, n, torch.float32) * 5.0)
        s["grads"].append(_matrices(g, b, m, n, kind))
    s["low"] = [x.bfloat16() for x in s["w"]]
    if own:
        from dropless_mixture_experts_warp_gb300 import muon
        s["plan"] = muon.plan(s["w"], s["grads"], copies=s["low"], m=s["m"], weight_decay=DECAY)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(state):
    kind = {"quantize": _run_quantize, "product": _run_product, "wgrad": _run_wgrad, "layer": _run_layer,
            "orthogonalize": _run_orthogonalize, "muon": _run_muon}
    return kind[state["case"]["op"]](state)


def _quantize_rows(x):
    """fp32 [R, C] -> E4M3 codes [R, C] and the scales of blocks of 128 along the rows, [ceil(C / 128), R]."""
    R, C = x.shape
    blocks = torch.nn.functional.pad(x, (0, -C % BLOCK)).view(R, -1, BLOCK)
    s = blocks.abs().amax(2).clamp_(min=FLOOR)
    s = s / torch.full_like(s, TOP)                                # by a tensor: rounded as a quotient
    codes = (blocks / s[:, :, None]).view(R, -1)[:, :C].to(E4M3)
    return codes.contiguous(), s.t().contiguous()


def _values_rows(codes, scales):
    R, C = codes.shape
    return codes.float() * scales.t().repeat_interleave(BLOCK, dim=1)[:, :C]


def _values_weights(codes, scales):
    E, N, K = codes.shape
    return codes.float() * scales.repeat_interleave(BLOCK, dim=1)[:, :N].repeat_interleave(BLOCK, dim=2)[:, :, :K]


def _run_quantize(s):
    both = s["case"]["both"]
    if own:
        from dropless_mixture_experts_warp_gb300 import fp8
        q = fp8.quantize(s["rows"], s["x"])
        return [q.codes, q.scales] + ([q.codes_t, q.scales_t] if both else [])
    x = s["x"].float()
    out = list(_quantize_rows(x))
    if both:                                                       # columns: the rows padded to whole blocks
        out += _quantize_rows(torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % BLOCK)).t())
    return out


def _places(s):
    """[E, cap] rows of every expert, and which of them are its own."""
    off = s["offsets"].long()
    at = torch.arange(s["cap"], device="cuda")[None] + off[:-1, None]
    return at.clamp(max=int(s["segments"][-1]) - 1), at < off[1:, None]


def _run_product(s):
    wide, E = s["case"]["wide"], s["case"]["E"]
    if own:
        from dropless_mixture_experts_warp_gb300 import fp8
        return fp8.matmul(s["a"], s["b"], s["out"], offsets=s["offsets"], transposed=wide)
    a, w = _values_rows(s["codes"], s["scales"]), _values_weights(s["w"], s["ws"])
    if not wide:
        w = w.transpose(1, 2)
    if E == 1:
        return (a @ w[0]).bfloat16()
    at, mine = _places(s)
    y = torch.bmm(a[at] * mine[:, :, None], w).bfloat16()
    return torch.zeros_like(s["out"]).index_put_((at[mine],), y[mine])


def _run_wgrad(s):
    if own:
        from dropless_mixture_experts_warp_gb300 import fp8
        return fp8.weight_grad(s["dy"], s["x"], s["out"], offsets=s["offsets"])
    dy, x = _values_rows(s["dy_t"], s["dy_s"]).t(), _values_rows(s["x_t"], s["x_s"]).t()
    if s["case"]["E"] == 1:
        return (dy.t() @ x)[None].bfloat16()
    at, mine = _places(s)
    return torch.bmm((dy[at] * mine[:, :, None]).transpose(1, 2), x[at] * mine[:, :, None]).bfloat16()


def _experts(x, gate, wgu, wd):
    """[B, rows, d] through the experts [B]: both products on quantised rows, G and U rounded to bf16 between."""
    B, n, d = x.shape
    f = wd.shape[2]
    xq = _values_rows(*_quantize_rows(x.reshape(B * n, d))).view(B, n, d)
    gu = torch.bmm(xq, wgu.transpose(1, 2)).bfloat16().float()
    g, u = gu[..., :f], gu[..., f:]
    h = gate[..., None] * (g / (1.0 + torch.exp(-g))) * u
    hq = _values_rows(*_quantize_rows(h.reshape(B * n, f))).view(B, n, f)
    return torch.bmm(hq, wd.transpose(1, 2)).bfloat16().float()


def _run_layer(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    if own:
        from dropless_mixture_experts_warp_gb300 import layer
        return layer.forward(s["b"], s["x"], s["logits"], None, None, weights_cached=True)
    val, top = torch.topk(s["logits"], k, dim=1)
    score = torch.exp(val - val[:, :1]) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-val))
    gate = score / score.sum(1, keepdim=True)
    x = s["x"].float()
    if T * k <= E:                                                 # few tokens: the chosen experts' weights alone
        e = top.reshape(-1)
        wgu, wd = (s[n].view(torch.uint8)[e].view(E4M3) for n in ("wgu", "wd"))
        y = _experts(x.repeat_interleave(k, 0)[:, None], gate.reshape(-1, 1), _values_weights(wgu, s["sgu"][e]),
                     _values_weights(wd, s["sd"][e]))
        return y.view(T, k, -1).sum(1).bfloat16()
    order = torch.argsort(top.reshape(-1), stable=True)
    e = top.reshape(-1)[order]
    place = torch.arange(T * k, device="cuda") - torch.searchsorted(e, e)
    xe = torch.zeros(E, s["cap"], c["d"], device="cuda").index_put_((e, place), x[order // k])
    ge = torch.zeros(E, s["cap"], device="cuda").index_put_((e, place), gate.reshape(-1)[order])
    y = _experts(xe, ge, _values_weights(s["wgu"], s["sgu"]), _values_weights(s["wd"], s["sd"]))
    rows = torch.empty(T * k, c["d"], device="cuda").index_put_((order,), y[e, place])
    return rows.view(T, k, -1).sum(1).bfloat16()


def _newton_schulz(x):
    """[b, m, n] -> the orthogonal factor's approximation, on the side with fewer rows."""
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / x.square().sum((1, 2), keepdim=True).sqrt().clamp(min=1e-30)
    for a, b, c in STEPS:
        A = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)
    return x.transpose(1, 2) if tall else x


def _run_orthogonalize(s):
    if own:
        from dropless_mixture_experts_warp_gb300 import muon
        return muon.orthogonalize([s["x"]], [s["out"]], s["plan"])
    return [_newton_schulz(s["x"].float()).bfloat16()]


def _run_muon(s):
    if own:
        from dropless_mixture_experts_warp_gb300 import muon
        muon.step(s["plan"], lr=LR, momentum=MOMENTUM, rms=RMS)
        return {"w": s["w"], "m": s["m"], "low": s["low"]}
    for w, m, grad, low in zip(s["w"], s["m"], s["grads"], s["low"]):
        m.mul_(MOMENTUM).add_(grad.float())
        o = _newton_schulz(grad.float() + MOMENTUM * m)
        w.sub_(LR * (DECAY * w + RMS * math.sqrt(max(w.shape[1:])) * o))
        low.copy_(w)
    return {"w": s["w"], "m": s["m"], "low": s["low"]}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"]
        out = _exact_codes(x)
        if case["both"]:
            pad = torch.zeros(-x.shape[0] % BLOCK, x.shape[1], dtype=x.dtype, device="cuda")
            out = out + _exact_codes(torch.cat([x, pad]).t().contiguous())
        return out
    if op == "product":
        rows, wide = s["codes"].shape[0], case["wide"]
        y = torch.zeros(rows, case["K"] if wide else case["N"], dtype=torch.float64, device="cuda")
        a = _exact_rows(s["codes"], s["scales"])
        for e in range(case["E"]):
            lo, hi = (0, rows) if case["E"] == 1 else (s["segments"][e], s["segments"][e + 1])
            if hi > lo:
                w = _exact_block(s["w"][e], s["ws"][e])
                y[lo:hi] = a[lo:hi] @ (w if wide else w.t())
        return y
    if op == "wgrad":
        dy, x = _exact_rows(s["dy_t"], s["dy_s"]), _exact_rows(s["x_t"], s["x_s"])
        if case["E"] == 1:
            return (dy @ x.t())[None]
        return torch.stack([dy[:, lo:hi] @ x[:, lo:hi].t() for lo, hi in zip(s["segments"], s["segments"][1:])])
    if op == "layer":
        return _exact_layer(s)
    if op == "orthogonalize":
        return [_exact_polar(s["x"].double())]
    shapes = _shapes(case)
    if sum(len(STEPS) * b * (4.0 * min(m, n) ** 2 * max(m, n) + 2.0 * min(m, n) ** 3) for b, m, n in shapes) > 1.5e13:
        return None
    out = {"w": [], "m": [], "low": []}
    for w, m, grad in zip(s["w"], s["m"], s["grads"]):
        m2 = MOMENTUM * m.double() + grad.double()
        o = _exact_polar(grad.double() + MOMENTUM * m2)
        w2 = w.double() * (1.0 - LR * DECAY) - LR * RMS * math.sqrt(max(w.shape[1:])) * o
        out["w"].append(w2), out["m"].append(m2), out["low"].append(w2)
    return out


def _exact_scale(amax):
    return (amax.clamp(min=FLOOR).double() / TOP).float().double()    # the scale is an fp32 number


def _exact_codes(x):
    R, C = x.shape
    codes, scales = [], []
    for lo in range(0, C, BLOCK):
        b = x[:, lo:lo + BLOCK].double()
        sc = _exact_scale(b.abs().amax(1).float())
        codes.append((b / sc[:, None]).to(E4M3))
        scales.append(sc)
    return [torch.cat([c.view(torch.uint8) for c in codes], 1).view(E4M3).double(), torch.stack(scales)]


def _exact_rows(codes, scales):
    out = codes.double()
    for i in range(scales.shape[0]):
        out[:, i * BLOCK:(i + 1) * BLOCK] *= scales[i].double()[:, None]
    return out


def _exact_block(codes, scales):
    n, k = codes.shape
    by_element = scales.double()[:, None, :, None].expand(-1, BLOCK, -1, BLOCK)
    return codes.double() * by_element.reshape(scales.shape[0] * BLOCK, -1)[:n, :k]


def _exact_through(v):
    """Rows of 64-bit values as their codes and scales stand for them (the values rounded to fp32 first)."""
    b = v.float().double().view(v.shape[0], -1, BLOCK)
    sc = _exact_scale(b.abs().amax(2).float())[:, :, None]
    return ((b / sc).to(E4M3).double() * sc).view(v.shape)


def _exact_layer(s):
    c = s["case"]
    T, d, f, E, k = (c[x] for x in ("T", "d", "f", "E", "k"))
    logits = s["logits"].double()
    top = torch.topk(logits, k, dim=1).indices
    p = torch.softmax(logits, 1) if c["score"] == "softmax" else torch.sigmoid(logits)
    p = torch.gather(p, 1, top)
    p = p / p.sum(1, keepdim=True)
    y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    x = _exact_through(s["x"].double())
    for e in top.unique().tolist():
        t, j = (top == e).nonzero(as_tuple=True)
        gu = (x[t] @ _exact_block(s["wgu"][e], s["sgu"][e]).t()).bfloat16().double()
        h = p[t, j, None] * gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]
        y.index_add_(0, t, (_exact_through(h) @ _exact_block(s["wd"][e], s["sd"][e]).t()).bfloat16().double())
    return y


def _exact_polar(x):
    out = torch.empty_like(x)
    for i in range(x.shape[0]):
        y = x[i] / torch.linalg.norm(x[i])
        for a, b, c in STEPS:
            if y.shape[0] <= y.shape[1]:
                A = y @ y.t()
                y = a * y + b * (A @ y) + c * (A @ (A @ y))
            else:
                A = y.t() @ y
                y = a * y + b * (y @ A) + c * ((y @ A) @ A)
        out[i] = y
    return out
