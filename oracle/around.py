"""Plain float64 forms of the operators around the layer (NumPy), for the tests.

Each gradient follows its formula; beside every result stands its majorant: the same
expression with every term taken by its absolute value, the scale of what rounding in fp32
can do to it.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24        # fp32: half a step, relative
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": U32}


def _act(g, sigmoid):
    """act(g) and its derivative."""
    if not sigmoid:
        return g, np.ones_like(g)
    a = 1.0 / (1.0 + np.exp(-g))
    return a, a / (1.0 + np.exp(g))    # 1 - a without the cancellation


def rms(h, eps):
    return 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)


def norm_fwd(h, w, eps, offset=0.0):
    return h * rms(h, eps) * (w + offset)


def _norm_grad(g, h, w, eps, offset):
    """Gradients of norm_fwd by h and w for the output gradient g, and their majorants."""
    r = rms(h, eps)
    n, hh = g * (w + offset), h * r
    dh = r * (n - hh * (n * hh).mean(axis=1, keepdims=True))
    m = r * (abs(n) + abs(hh) * abs(n * hh).mean(axis=1, keepdims=True))
    return dh, m, (g * hh).sum(axis=0), abs(g * hh).sum(axis=0)


def norm_bwd(dx, h, w, eps, offset=0.0, dh_add=None):
    dh, m, dw, mw = _norm_grad(dx, h, w, eps, offset)
    if dh_add is not None:
        dh, m = dh + dh_add, m + abs(dh_add)
    return {"dh": (dh, m), "dw": (dw, mw)}


def _gate(gate, kind, sigmoid):
    if kind == "none":
        return 1.0, 0.0
    a, da = _act(gate, sigmoid)
    return (a[None, :], da[None, :]) if kind == "channel" else (a[:, None], da[:, None])


def merge_fwd(h, y, w_post, gate, w_next, *, eps, kind="none", sigmoid=False, offset=0.0, alpha=1.0, beta=1.0):
    z = y if w_post is None else norm_fwd(y, w_post, eps, offset)
    a, _ = _gate(gate, kind, sigmoid)
    out = alpha * h + beta * a * z
    m = abs(alpha * h) + abs(beta * a * z)
    res = {"h_out": (out, m)}
    if w_next is not None:
        r = rms(out, eps)
        x = out * r * (w_next + offset)
        # an error of m * u in the stream reaches x through the element and through r
        mx = m * r * abs(w_next + offset) + abs(x) * (1.0 + r * r * (m * abs(out)).mean(axis=1, keepdims=True))
        res["x"] = (x, mx)
    return res


def merge_bwd(dh_out, dx, h_out, y, w_post, gate, w_next, *, eps, kind="none", sigmoid=False, offset=0.0, alpha=1.0,
              beta=1.0):
    res = {}
    T, d = (dh_out if dh_out is not None else dx).shape
    D = np.zeros((T, d)) if dh_out is None else dh_out
    m = abs(D)
    if w_next is not None:
        more, mm, dw, mw = _norm_grad(dx, h_out, w_next, eps, offset)
        D, m = D + more, m + mm
        res["dw_next"] = (dw, mw)
    res["dh"] = (alpha * D, abs(alpha) * m)
    a, da = _gate(gate, kind, sigmoid)
    dz, mz = beta * a * D, abs(beta * a) * m
    z = y
    if w_post is not None:
        z = norm_fwd(y, w_post, eps, offset)
        dy, _, dw, _ = _norm_grad(dz, y, w_post, eps, offset)
        _, md, _, mw = _norm_grad(mz, abs(y), abs(w_post + offset), eps, 0.0)
        res["dy"], res["dw_post"] = (dy, md), (dw, mw)
    else:
        res["dy"] = (dz, mz)
    if kind != "none":
        axis = 0 if kind == "channel" else 1
        res["dgate"] = ((beta * da * D * z).sum(axis=axis), (abs(beta * da * z) * m).sum(axis=axis))
    return res


# ------------------------------------------------------------------ balance loss

def probabilities(l, score):
    """[T, E] logits -> p: the softmax of the scores' logarithms (log sigmoid(l) = -log(1 + e^-l), or l itself); a
    row of -inf gives p = 0."""
    g = l if score == "softmax" else -np.logaddexp(0.0, -l)
    top = g.max(axis=1, keepdims=True)
    e = np.exp(g - np.where(np.isneginf(top), 0.0, top))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def logsumexp(l):
    top = l.max(axis=1)
    top = np.where(np.isneginf(top), 0.0, top)
    s = np.exp(l - top[:, None]).sum(axis=1)
    return np.where(s > 0, top + np.log(np.where(s > 0, s, 1.0)), 0.0)


def balance_fwd(l, idx, offsets, mask, k, score, coef, z_coef):
    E, S = l.shape[1], len(offsets) - 1
    counts, mean, n = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    loss, z = 0.0, 0.0
    for s in range(S):
        t = np.arange(offsets[s], offsets[s + 1])
        if mask is not None:
            t = t[mask[t] != 0]
        n[s] = len(t)
        if not len(t):
            continue
        counts[s] = np.bincount(idx[t].ravel(), minlength=E)
        mean[s] = probabilities(l[t], score).mean(axis=0)
        loss += (E * counts[s] / (k * n[s]) * mean[s]).sum()
        z += (logsumexp(l[t]) ** 2).sum()
    return {"losses": np.array([coef * loss / max(1, (n > 0).sum()), z_coef * z / max(1, n.sum())]), "counts": counts,
            "prob_mean": mean, "seq_tokens": n}


def balance_bwd(l, offsets, mask, counts, n, k, score, coef, z_coef, grad=(1.0, 1.0)):
    """Gradient by the logits and its majorant."""
    out, maj = np.zeros_like(l), np.zeros_like(l)
    E = l.shape[1]
    for s in range(len(offsets) - 1):
        t = np.arange(offsets[s], offsets[s + 1])
        if mask is not None:
            t = t[mask[t] != 0]
        if not len(t):
            continue
        x = l[t]
        p, q = probabilities(x, score), probabilities(x, "softmax")
        f = E * counts[s] / (k * n[s])
        g = grad[0] * coef / (n > 0).sum() / n[s]
        m = (f * p).sum(axis=1, keepdims=True)
        d, md = g * p * (f - m), abs(g) * p * (f + m)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                d, md = d / (1 + np.exp(x)), md / (1 + np.exp(x))
        zz = grad[1] * z_coef * 2 / n.sum() * logsumexp(x)[:, None] * q
        out[t], maj[t] = d + zz, md + abs(zz)
    return out, maj


# ------------------------------------------------------------------ AdamW

ADAM_BLOCK = 128


def adamw(w, g, m, v, *, t, lr, beta1, beta2, eps, wd, grad_scale=1.0):
    """One step in float64: new w, m, v."""
    g = grad_scale * g
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    w = w - lr * (m / (1 - beta1 ** t) / (np.sqrt(v / (1 - beta2 ** t)) + eps) + wd * w)
    return w, m, v


def _mix(x):
    x = x.astype(np.uint32)
    x ^= x >> np.uint32(16)
    x *= np.uint32(0x6A09E667)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0xBB67AE85)
    return x ^ (x >> np.uint32(16))


def adamw_draws(seed, t, tensor, n, first=0):
    """The two numbers in (0, 1) that draw the codes of elements first .. first + n of a tensor."""
    i = np.arange(first, first + n, dtype=np.uint64)
    low, high = i.astype(np.uint32), (i >> np.uint64(32)).astype(np.uint32)
    with np.errstate(over="ignore"):
        base = _mix(_mix(np.array([seed], np.uint32)) + np.uint32(t))
        key = _mix(base + np.array([tensor], np.uint32) * np.uint32(0x6A09E667) + high * np.uint32(0xBB67AE85))
        u = _mix(low * np.uint32(0x9E3779B9) + key)
    return ((u & np.uint32(0xFFFF)) + 0.5) / 65536, ((u >> np.uint32(16)) + 0.5) / 65536


def block_scales(x):
    """Largest |x| of each block of 128 (the last may be shorter); 0 below fp32's normal numbers."""
    pad = np.zeros(-(-len(x) // ADAM_BLOCK) * ADAM_BLOCK)
    pad[:len(x)] = abs(x)
    s = pad.reshape(-1, ADAM_BLOCK).max(axis=1)
    return np.where(s < np.finfo(np.float32).tiny, 0.0, s)


def encode(x, scales, draws, top, power):
    """Codes of x (signed for power 2, unsigned for power 4), and the distance of the draw from the border between
    the two codes around x, as a share of their distance."""
    s = np.repeat(scales, ADAM_BLOCK)[:len(x)]
    share = np.divide(abs(x), s, out=np.zeros_like(x), where=s > 0)
    k = np.floor(np.minimum(share, 1.0) ** (1.0 / power) * top * (1 + 1e-13))
    lo, hi = (k / top) ** power, ((k + 1) / top) ** power
    chance = (share - lo) / (hi - lo)
    code = np.minimum(k + (draws < chance), top)
    if power == 4:
        code = np.where(share > 0, np.maximum(code, 1), code)
    return (np.sign(x) * code).astype(np.int64), abs(draws - chance)


def decode(code, scales, top, power):
    s = np.repeat(scales, ADAM_BLOCK)[:len(code)]
    return np.sign(code) * s * (abs(code) / top) ** power
