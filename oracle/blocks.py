"""float64 forms of the 8-bit products with blocks of 128 and of the orthogonalised update (test infrastructure)."""
import numpy as np
import torch

BLOCK = 128
TOP, FLOOR = 448.0, 2.0 ** -64
E4M3 = torch.float8_e4m3fn
BF16_HALF, U32 = 2.0 ** -8, 2.0 ** -24


def up(n):
    return -(-n // BLOCK) * BLOCK


def scale_of(amax):
    """The fp32 scale of blocks whose largest magnitudes (float32) are given."""
    amax = np.maximum(amax.astype(np.float32), np.float32(FLOOR))
    return (amax / np.float32(TOP)).astype(np.float32)


def _codes(x, s):
    """E4M3 of the fp32 quotients; either zero is code 0."""
    with np.errstate(invalid="ignore"):
        q = ((x.astype(np.float32) + np.float32(0)) / s.astype(np.float32)).astype(np.float32)
    return torch.from_numpy(np.ascontiguousarray(q)).to(E4M3)


def quantize_rows(x):
    """x [R, C] -> codes [R, C] (E4M3 tensor), scales [ceil(C / 128), R] float32."""
    R, C = x.shape
    p = np.zeros((R, up(C)), dtype=np.float32)
    p[:, :C] = x
    s = scale_of(np.abs(p.reshape(R, -1, BLOCK)).max(2))
    return _codes(p, np.repeat(s, BLOCK, 1))[:, :C].contiguous(), np.ascontiguousarray(s.T)


def quantize_columns(x):
    """x [R, C] -> codes_t [C, R up to 128], scales_t [ceil(R / 128), C]."""
    p = np.zeros((up(x.shape[0]), x.shape[1]), dtype=np.float32)
    p[:x.shape[0]] = x
    return quantize_rows(p.T)


def quantize_weights(w):
    """w [E, N, K] -> codes [E, N, K], scales [E, ceil(N / 128), ceil(K / 128)]."""
    E, N, K = w.shape
    p = np.zeros((E, up(N), up(K)), dtype=np.float32)
    p[:, :N, :K] = w
    s = scale_of(np.abs(p.reshape(E, up(N) // BLOCK, BLOCK, up(K) // BLOCK, BLOCK)).max((2, 4)))
    return _codes(p, s.repeat(BLOCK, 1).repeat(BLOCK, 2))[:, :N, :K].contiguous(), s


def rows_values(codes, scales):
    """What codes [R, C] with scales [ceil(C / 128), R] stand for, float64."""
    c = codes.double().numpy()
    return c * np.repeat(np.asarray(scales, np.float64).T, BLOCK, 1)[:, :c.shape[1]]


def weights_values(codes, scales):
    c = codes.double().numpy()
    s = np.asarray(scales, np.float64).repeat(BLOCK, 1).repeat(BLOCK, 2)
    return c * s[:, :c.shape[1], :c.shape[2]]


def product(a, w, offsets=None):
    """a [R, K] times each expert's w [E, N, K]^T, and the sum of magnitudes; rows outside the offsets NaN."""
    R, N = a.shape[0], w.shape[1]
    offsets = [0, R] if offsets is None else offsets
    y, mag = np.full((R, N), np.nan), np.zeros((R, N))
    for e in range(w.shape[0]):
        lo, hi = min(offsets[e], R), min(offsets[e + 1], R)
        y[lo:hi] = a[lo:hi] @ w[e].T
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w[e]).T
    return y, mag


def weight_grad(dy, x, offsets=None):
    offsets = [0, dy.shape[0]] if offsets is None else offsets
    out = [(dy[lo:hi].T @ x[lo:hi], np.abs(dy[lo:hi]).T @ np.abs(x[lo:hi])) for lo, hi in zip(offsets, offsets[1:])]
    return np.stack([o[0] for o in out]), np.stack([o[1] for o in out])


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def swiglu(g, u, w):
    return w[:, None] * g * sigmoid(g) * u


def swiglu_bwd(g, u, w, dh):
    """-> dG, dU, dw."""
    s = sigmoid(g)
    silu, da = g * s, w[:, None] * dh
    return da * u * s * (1 + g * (1 - s)), da * silu, (silu * u * dh).sum(1)


COEFFICIENTS = [(3.4445, -4.7750, 2.0315)] * 5


def newton_schulz(x, coefficients=COEFFICIENTS, eps=0.0):
    """x [m, n] float64 -> a_i X + b_i X X^T X + c_i X X^T X X^T X, step by step, from X / max(|X|_F, eps)."""
    n = max(np.linalg.norm(x), eps)
    x = x / n if n > 0 else np.zeros_like(x)
    for a, b, c in coefficients:
        x3 = x @ (x.T @ x) if x.shape[0] > x.shape[1] else (x @ x.T) @ x
        x5 = x3 @ (x.T @ x) if x.shape[0] > x.shape[1] else (x @ x.T) @ x3
        x = a * x + b * x3 + c * x5
    return x


def muon_step(w, m, grad, lr, momentum, decay, rms, nesterov=True, coefficients=COEFFICIENTS, eps=0.0):
    """One matrix: (w', m', update)."""
    m = momentum * m + grad
    o = newton_schulz(grad + momentum * m if nesterov else m, coefficients, eps)
    return w - lr * (decay * w + rms * np.sqrt(max(w.shape)) * o), m, o


def newton_schulz_rounded(x, coefficients=COEFFICIENTS, eps=0.0):
    """newton_schulz as the kernels round it: products on fp16 operands, X in two parts in the addend, multiples of I
    taken off A and B in the last two steps, everything else exact.  How far it is from newton_schulz is what that arithmetic costs."""
    h = lambda v: v.astype(np.float16).astype(np.float64)  # noqa: E731
    x = x.T if x.shape[0] > x.shape[1] else x
    n = max(np.linalg.norm(x), eps)
    length = up(x.shape[1])
    scale = 1.0
    while scale * scale * 4 <= length:
        scale *= 2
    x = scale * x / n if n > 0 else np.zeros_like(x)
    hi = h(x)
    lo = h(x - hi)
    for k, (a, b, c) in enumerate(coefficients):
        late = k >= 1 and k >= len(coefficients) - 2
        u, t, eye = 0.5 * late, (a - 1) * late, np.eye(x.shape[0])
        A = h(hi @ hi.T / scale ** 2 - u * eye)
        B = h(c * (A @ A) + (b + 2 * u * c) * A + (b * u + c * u * u + t) * eye)
        v = (a - t) * (hi + lo) + B @ hi
        hi = h(v)
        lo = h(v - hi)
    return hi / scale


def newton_schulz_split(x, coefficients=COEFFICIENTS, eps=0.0, step=2.0 ** -23):
    """newton_schulz as the kernels round it with operands in two fp16 parts, and with what their fp32 sums may lose: at
    every step of 16 along a contraction up to a unit in the last place of the largest value that the sum reaches, here
    always towards 0 (step=0: the operands' roundings alone)."""
    def two(v):
        hi = v.astype(np.float16).astype(np.float64)
        return hi, (v - hi).astype(np.float16).astype(np.float64)

    def product(a, b):
        v = a[0] @ b[0] + a[0] @ b[1] + a[1] @ b[0]
        lost = (-(-a[0].shape[1] // 16) + 2) * step
        return v - np.sign(v) * np.minimum(lost * (np.abs(a[0]) @ np.abs(b[0])), np.abs(v)) if step else v

    x = x.T if x.shape[0] > x.shape[1] else x
    n = max(np.linalg.norm(x), eps)
    length = up(x.shape[1])
    scale = 1.0
    while scale * scale * 4 <= length:
        scale *= 2
    x = two(scale * x / n if n > 0 else np.zeros_like(x))
    for k, (a, b, c) in enumerate(coefficients):
        late = k >= 1 and k >= len(coefficients) - 2
        u, t, eye = 0.5 * late, (a - 1) * late, np.eye(x[0].shape[0])
        A = two(product(x, (x[0].T, x[1].T)) / scale ** 2 - u * eye)
        B = two(c * product(A, A) + (b + 2 * u * c) * (A[0] + A[1]) + (b * u + c * u * u + t) * eye)
        x = two((a - t) * (x[0] + x[1]) + product(B, x))
    return (x[0] + x[1]) / scale
