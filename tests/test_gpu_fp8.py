"""The 8-bit products with blocks of 128 on the GPU, against float64 on the CPU.

Codes and scales are compared bit for bit.  Products: one rounding to bf16 (2^-8 of the value), and fp32 sums, each
of the K products and of the scaled block sums adding at most 2^-24 of the sum of magnitudes so far; tensor cores
may drop what is below 2^-24 of the largest term of a step instead of rounding, so every term counts twice.
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from oracle import blocks as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def bf16(rng, *shape, scale=1.0):
    x = rng.standard_normal(shape) * scale
    return torch.from_numpy(x).to(torch.bfloat16)


def activations(rng, R, C):
    x = rng.standard_normal((R, C)) * (0.3 + rng.random((R, 1)))
    x[:, :: max(1, C // 5)] *= 30.0
    if R > 2:
        x[R // 2] = 0.0
    if C > 40 and R > 1:
        x[1, :40] *= 1e-30
    return torch.from_numpy(x).to(torch.bfloat16)


def same_codes(got, ref):
    assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))


def close(got, ref, mag, terms):
    got = got.double().cpu().numpy()
    bound = ob.BF16_HALF * np.abs(ref) + (1 + ob.BF16_HALF) * 2 * (terms + 2) * ob.U32 * mag + 1e-37
    off = np.abs(got - ref)
    assert np.all(off <= bound), (np.max(off - bound), np.abs(ref).max())


# ------------------------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("R,C", [(1, 16), (1, 7168), (3, 128), (5, 272), (127, 144), (128, 256), (129, 400), (1000, 2048)])
@pytest.mark.parametrize("both", [False, True])
def test_quantize(R, C, both):
    from dropless_mixture_experts_warp_gb300 import fp8
    x = activations(np.random.default_rng(R * 7 + C), R, C)
    a = fp8.quantize(fp8.allocate_rows(R, C, both=both), x.cuda())
    codes, scales = ob.quantize_rows(x.float().numpy())
    same_codes(a.codes, codes)
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    if both:
        codes, scales = ob.quantize_columns(x.float().numpy())
        same_codes(a.codes_t, codes)
        assert np.array_equal(a.scales_t.cpu().numpy(), scales)


def test_quantize_every_quotient():
    """All bf16 magnitudes of seven binades under 64 scales: the corrected quotients give the codes of exact division."""
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(3)
    tops = rng.integers(0x3F80, 0x4380, 64)                       # the largest value of each row, 1 to 256
    bits = np.empty((64, 1024), dtype=np.int64)
    for i, top in enumerate(tops):
        bits[i] = rng.integers(max(0, top - 7 * 128), top + 1, 1024)
        bits[i, :: 128] = top
    x = torch.from_numpy((bits | (rng.integers(0, 2, bits.shape) << 15)).astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    a = fp8.quantize(fp8.allocate_rows(64, 1024, both=True), x.cuda())
    codes, scales = ob.quantize_rows(x.float().numpy())
    same_codes(a.codes, codes)
    assert np.array_equal(a.scales.cpu().numpy(), scales)


def test_quantize_extremes():
    """Zeros, values under the floor, the largest finite values, NaN and infinities."""
    from dropless_mixture_experts_warp_gb300 import fp8
    x = torch.zeros(6, 256, dtype=torch.bfloat16)
    x[1, :5] = torch.tensor([1e-30, -1e-25, 1e-38, 0.0, -0.0])
    x[2, :3] = torch.tensor([3.3e38, -3.3e38, 1.0])
    x[3, 7], x[3, 8] = float("nan"), 2.0
    x[4, 9], x[4, 10] = float("inf"), 2.0
    x[5, 200] = 1.0
    a = fp8.quantize(fp8.allocate_rows(6, 256, both=True), x.cuda())
    v = a.codes.float().cpu() * a.scales.cpu().t().repeat_interleave(128, 1)
    ref = ob.quantize_rows(x.float().numpy())[0].view(torch.uint8)
    assert torch.equal(a.codes.view(torch.uint8).cpu()[[0, 1, 2, 5]], ref[[0, 1, 2, 5]])
    assert torch.isfinite(v[[0, 1, 2, 5]]).all() and v[2, 0] > 3.2e38
    assert torch.isnan(v[3, 7]) and v[3, 8] == 2.0 and torch.isfinite(v[3, :7]).all()
    assert torch.isnan(v[4, :128]).all() and torch.isfinite(v[4, 128:]).all()


def test_quantize_gathered_rows():
    """Rows through a map (negative: zeros), and 128-row blocks from n_rows on left as they were."""
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(5)
    x = activations(rng, 37, 272)
    mp = torch.from_numpy(rng.integers(-1, 37, 384).astype(np.int32))
    n = torch.tensor([256], dtype=torch.int32).cuda()
    full = torch.where(mp[:, None] >= 0, x.float()[mp.clamp(min=0).long()], 0.0).numpy()
    rc, rs = ob.quantize_rows(full)
    cc, cs = ob.quantize_columns(full)
    for both in (False, True):
        a = fp8.allocate_rows(384, 272, both=both)
        for t in (a.codes, a.scales, a.codes_t, a.scales_t):
            if t is not None:
                t.view(torch.uint8).fill_(0x11)
        fp8.quantize(a, x.cuda(), row_map=mp.cuda(), n_rows=n)
        same_codes(a.codes[:256], rc[:256])
        assert np.array_equal(a.scales[:, :256].cpu().numpy(), rs[:, :256])
        assert (a.codes[256:].view(torch.uint8) == 0x11).all() and (a.scales[:, 256:].contiguous().view(torch.uint8) == 0x11).all()
        if both:
            same_codes(a.codes_t[:, :256].contiguous(), cc[:, :256].contiguous())
            assert np.array_equal(a.scales_t[:2].cpu().numpy(), cs[:2])
            assert (a.codes_t[:, 256:].contiguous().view(torch.uint8) == 0x11).all() and (a.scales_t[2:].view(torch.uint8) == 0x11).all()


@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (2, 128, 256), (3, 144, 400), (1, 2064, 1456)])
def test_quantize_weights(E, N, K):
    from dropless_mixture_experts_warp_gb300 import fp8
    w = bf16(np.random.default_rng(N + K), E, N, K, scale=0.02)
    q = fp8.quantize_weights(fp8.allocate_weights(E, N, K, both=True), w.cuda())
    codes, scales = ob.quantize_weights(w.float().numpy())
    same_codes(q.codes, codes)
    same_codes(q.codes_t, codes.transpose(1, 2).contiguous())
    assert np.array_equal(q.scales.cpu().numpy(), scales)


# ------------------------------------------------------------------------------------ products

def rows(rng, R, C, both=False):
    x = activations(rng, R, C).float().numpy()
    codes, scales = ob.quantize_rows(x)
    return codes, scales


def weights(rng, E, N, K):
    codes = torch.from_numpy((rng.standard_normal((E, N, K)) * 100).clip(-448, 448).astype(np.float32)).to(ob.E4M3)
    scales = ((0.5 + rng.random((E, ob.up(N) // 128, ob.up(K) // 128))) * 1e-3).astype(np.float32)
    return codes, scales


def cuda(x):
    return (x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))).cuda()


@pytest.mark.parametrize("R,N,K", [(1, 16, 16), (1, 4096, 7168), (5, 128, 128), (127, 144, 272), (128, 256, 256), (129, 272, 400),
                                   (300, 2064, 1456), (1237, 640, 144),
                                   (5, 4096, 2064), (130, 272, 1040), (64, 16, 4096), (17, 1040, 7168)])
@pytest.mark.parametrize("transposed", [False, True])
def test_product(R, N, K, transposed):
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(R + N + K)
    codes, scales = rows(rng, R, N if transposed else K)
    wc, ws = weights(rng, 1, N, K)
    w = fp8.weights_of(cuda(wc), cuda(ws), cuda(wc.transpose(1, 2).contiguous()) if transposed else None)
    a = fp8.rows_of(cuda(codes), cuda(scales))
    out = torch.full((R, K if transposed else N), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.matmul(a, w, out, transposed=transposed)
    fp8.check(a)
    v = ob.weights_values(wc, ws)
    ref, mag = ob.product(ob.rows_values(codes, scales), v.transpose(0, 2, 1) if transposed else v)
    close(out, ref, mag, N if transposed else K)


COUNTS = [[1], [0, 5, 0], [128, 0, 1, 130, 257], [0, 0], [3] * 40]


def segments(counts):
    off = [0]
    for n in counts:
        off.append(off[-1] + ob.up(n))
    return off


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K,transposed", [(256, 384, False), (144, 272, False), (400, 256, True)])
def test_grouped_product(counts, N, K, transposed):
    """Ragged experts, some without rows; rows behind the last segment stay as they were."""
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(len(counts) + N)
    off = segments(counts)
    R, E = off[-1] + 200, len(counts)
    codes, scales = rows(rng, R, N if transposed else K)
    wc, ws = weights(rng, E, N, K)
    w = fp8.weights_of(cuda(wc), cuda(ws), cuda(wc.transpose(1, 2).contiguous()) if transposed else None)
    a = fp8.rows_of(cuda(codes), cuda(scales))
    out = torch.full((R, K if transposed else N), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.matmul(a, w, out, offsets=torch.tensor(off, dtype=torch.int32).cuda(), transposed=transposed)
    fp8.check(a)
    v = ob.weights_values(wc, ws)
    ref, mag = ob.product(ob.rows_values(codes, scales), v.transpose(0, 2, 1) if transposed else v, off)
    n = off[-1]
    close(out[:n], ref[:n], mag[:n], N if transposed else K)
    assert (out[n:] == 7.0).all()


@pytest.mark.parametrize("counts", [[5000], [1300, 0, 640, 1, 129, 3000, 257], [0, 0, 5000, 128, 0], [4000] + [100] * 9 + [1024]])
@pytest.mark.parametrize("N,K,transposed", [(1040, 144, False), (1296, 400, False), (528, 1296, True)])
def test_product_of_many_rows(counts, N, K, transposed):
    """Tiles of 256 rows and columns: experts with odd numbers of 128 rows, ends inside a tile, none at all."""
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(sum(counts) + N)
    off = segments(counts)
    R, E = off[-1] + 130, len(counts)
    codes, scales = rows(rng, R, N if transposed else K)
    wc, ws = weights(rng, E, N, K)
    w = fp8.weights_of(cuda(wc), cuda(ws), cuda(wc.transpose(1, 2).contiguous()) if transposed else None)
    a = fp8.rows_of(cuda(codes), cuda(scales))
    out = torch.full((R, K if transposed else N), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.matmul(a, w, out, offsets=torch.tensor(off, dtype=torch.int32).cuda(), transposed=transposed)
    fp8.check(a)
    v = ob.weights_values(wc, ws)
    ref, mag = ob.product(ob.rows_values(codes, scales), v.transpose(0, 2, 1) if transposed else v, off)
    n = off[-1]
    close(out[:n], ref[:n], mag[:n], N if transposed else K)
    assert (out[n:] == 7.0).all()


def test_product_of_many_rows_one_matrix():
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(4)
    R, N, K = 4997, 1040, 272
    codes, scales = rows(rng, R, K)
    wc, ws = torch.from_numpy(rng.standard_normal((1, N, K)).astype(np.float32)).to(ob.E4M3), (0.5 + rng.random((1, 9, 3))).astype(np.float32)
    a, w = fp8.rows_of(cuda(codes), cuda(scales)), fp8.weights_of(cuda(wc), cuda(ws))
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    fp8.matmul(a, w, out)
    fp8.check(a)
    ref, mag = ob.product(ob.rows_values(codes, scales), ob.weights_values(wc, ws), [0, R])
    close(out, ref, mag, K)


@pytest.mark.parametrize("counts", COUNTS + [[300]])
@pytest.mark.parametrize("N,K", [(16, 16), (256, 384), (144, 272), (400, 1040)])
def test_weight_grad(counts, N, K):
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(len(counts) + N)
    off = segments(counts)
    R, E = off[-1], len(counts)
    if R == 0:
        R = 128
    dy, x = activations(rng, R, N).float().numpy(), activations(rng, R, K).float().numpy()
    (dc, ds), (xc, xs) = ob.quantize_columns(dy), ob.quantize_columns(x)
    da, xa = fp8.rows_of(codes_t=cuda(dc), scales_t=cuda(ds)), fp8.rows_of(codes_t=cuda(xc), scales_t=cuda(xs))
    out = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.weight_grad(da, xa, out, offsets=torch.tensor(off, dtype=torch.int32).cuda())
    fp8.check(da)
    ref, mag = ob.weight_grad(ob.rows_values(dc, ds).T, ob.rows_values(xc, xs).T, off)
    close(out, ref, mag, max(counts))


# ------------------------------------------------------------------------------------ SwiGLU

def stands_for(codes, scales, ref, mag=None):
    """Codes and scales stand for ref within half a step of E4M3 (2^-4 of the value; 2^-10 of the scale among its
    subnormals), the values computed in fp32 with exponentials good to 2^-20 of `mag` (default: of the value)."""
    mag = np.abs(ref) if mag is None else mag

    def top(a):
        p = np.zeros((a.shape[0], ob.up(a.shape[1])))
        p[:, :a.shape[1]] = a
        return p.reshape(a.shape[0], -1, 128).max(2)

    v = ob.rows_values(codes.cpu(), scales.cpu().numpy())
    s = np.maximum(top(np.abs(ref)), ob.FLOOR) / ob.TOP
    off = np.abs(scales.cpu().numpy().T - s) - (2.0 ** -18 * top(mag) / ob.TOP + 2.0 ** -23 * s)
    assert np.all(off <= 0), np.max(off)
    s = np.repeat(s, 128, 1)[:, :ref.shape[1]]
    off = np.abs(v - ref) - (np.abs(ref) * 2.0 ** -4 + s * 2.0 ** -10 + 2.0 ** -16 * mag + 2.0 ** -17 * s)
    assert np.all(off <= 0), np.max(off)


def gradient_terms(g, u, w, dh):
    """Sums of magnitudes of dG | dU: silu' = s (1 + g (1 - s)) is 0 near g = -1.28, where its terms cancel, so that dG is
    exact to a part of s (1 + |g| (1 - s)) only."""
    s, da = ob.sigmoid(g), np.abs(w[:, None] * dh)
    return np.concatenate([da * np.abs(u) * s * (1 + np.abs(g) * (1 - s)), da * np.abs(g) * s], 1)


@pytest.mark.parametrize("R,f", [(1, 16), (5, 272), (129, 128), (300, 640)])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu(R, f, weighted):
    from dropless_mixture_experts_warp_gb300 import binding as B, fp8
    rng = np.random.default_rng(R + f)
    gu = bf16(rng, R, 2 * f, scale=3.0)
    gu[0, :4] = torch.tensor([90.0, -90.0, 300.0, -300.0])
    w = torch.from_numpy(rng.random(R).astype(np.float32)) if weighted else None
    h = fp8.allocate_rows(R, f)
    B.moe_fp8_swiglu(gu.cuda(), None if w is None else w.cuda(), R, f, None, h.codes, h.scales)
    v = gu.double().numpy()
    ref = ob.swiglu(v[:, :f], v[:, f:], np.ones(R) if w is None else w.double().numpy())
    stands_for(h.codes, h.scales, ref)


@pytest.mark.parametrize("R,f,used", [(1, 128, None), (130, 256, None), (512, 384, 384), (256, 1024, 0)])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu_gradient(R, f, used, weighted):
    from dropless_mixture_experts_warp_gb300 import binding as B, fp8
    rng = np.random.default_rng(R + f)
    gu, dh = bf16(rng, R, 2 * f, scale=2.0), bf16(rng, R, f, scale=0.1)
    gu[0, :4] = torch.tensor([90.0, -90.0, 300.0, -300.0])
    w = torch.from_numpy(rng.random(R).astype(np.float32)) if weighted else None
    dgu, h = fp8.allocate_rows(R, 2 * f, both=True), fp8.allocate_rows(R, f, both=True)
    dw, part = (torch.full((R,), 7.0, device="cuda"), torch.empty(R, f // 128, device="cuda")) if weighted else (None, None)
    for t in (dgu.codes, dgu.codes_t, h.codes_t):
        t.view(torch.uint8).fill_(0x11)
    for t in (dgu.scales, dgu.scales_t, h.scales_t):
        t.fill_(7.0)
    n = None if used is None else torch.tensor([used], dtype=torch.int32).cuda()
    B.moe_fp8_swiglu_bwd(gu.cuda(), dh.cuda(), None if w is None else w.cuda(), R, f, n, dgu.codes, dgu.scales, dgu.codes_t,
                         dgu.scales_t, h.codes_t, h.scales_t, dw, part)
    k = R if used is None else used
    v, d = gu.double().numpy()[:k], dh.double().numpy()[:k]
    ww = np.ones(k) if w is None else w.double().numpy()[:k]
    dG, dU, dws = ob.swiglu_bwd(v[:, :f], v[:, f:], ww, d)
    ref, hr = np.concatenate([dG, dU], 1), ob.swiglu(v[:, :f], v[:, f:], ww)
    if k:
        mag = gradient_terms(v[:, :f], v[:, f:], ww, d)
        stands_for(dgu.codes[:k], dgu.scales[:, :k], ref, mag)
        pad = np.zeros((ob.up(k) - k, 2 * f))
        kt = ob.up(k)
        stands_for(dgu.codes_t[:, :kt], dgu.scales_t[: kt // 128], np.concatenate([ref, pad]).T, np.concatenate([mag, pad]).T)
        stands_for(h.codes_t[:, :kt], h.scales_t[: kt // 128], np.concatenate([hr, pad[:, :f]]).T)
        if weighted:
            s = ob.sigmoid(v[:, :f])
            mag = np.abs(v[:, :f] * s * v[:, f:] * d).sum(1)
            assert np.all(np.abs(dw[:k].double().cpu().numpy() - dws) <= (f + 64) * ob.U32 * mag + 1e-30)
    if used is not None:
        assert (dgu.codes[k:].view(torch.uint8) == 0x11).all() and (dgu.scales[:, k:] == 7.0).all()
        assert (h.codes_t[:, k:].contiguous().view(torch.uint8) == 0x11).all() and (h.scales_t[k // 128:] == 7.0).all()


@pytest.mark.parametrize("offsets", [[0, 256, 128], [128, 256, 384], [0, 100, 256], [0, -128, 256], [-128, 0, 128]])
def test_offsets_out_of_order(offsets):
    from dropless_mixture_experts_warp_gb300 import binding as B, fp8
    rng = np.random.default_rng(5)
    o = torch.tensor(offsets, dtype=torch.int32).cuda()
    a, x = (fp8.quantize(fp8.allocate_rows(384, C, both=True), activations(rng, 384, C).cuda()) for C in (144, 256))
    w = fp8.weights_of(*map(cuda, weights(rng, 2, 272, 144)))
    out, grad = torch.full((384, 272), 7.0, device="cuda").bfloat16(), torch.full((2, 144, 256), 7.0, device="cuda").bfloat16()
    for call in (lambda: fp8.matmul(a, w, out, o), lambda: fp8.weight_grad(a, x, grad, o)):
        call()
        with pytest.raises(B.MoeError) as e:
            fp8.check(a)
        assert e.value.status == 7
        a.status.zero_()
    assert (out == 7.0).all() and (grad == 0.0).all()


def test_swiglu_gradient_of_rows_that_weigh_nothing():
    """A row of weight 0 is zeros in all forms, infinities and NaN in it included; columns keep the other rows' scales."""
    from dropless_mixture_experts_warp_gb300 import binding as B, fp8
    R, f = 130, 256
    rng = np.random.default_rng(8)
    gu, dh, w = bf16(rng, R, 2 * f), bf16(rng, R, f), torch.rand(R) + 0.5
    none = [0, 77, 129]
    w[none] = 0.0
    got = []
    for fill in (0.0, float("inf"), float("nan")):
        g, d = gu.clone(), dh.clone()
        g[none], d[none] = fill, fill
        dgu, h = fp8.allocate_rows(R, 2 * f, both=True), fp8.allocate_rows(R, f, both=True)
        dw, part = torch.empty(R, device="cuda"), torch.empty(R, f // 128, device="cuda")
        B.moe_fp8_swiglu_bwd(g.cuda(), d.cuda(), w.cuda(), R, f, None, dgu.codes, dgu.scales, dgu.codes_t, dgu.scales_t, h.codes_t, h.scales_t,
                             dw, part)
        keep = [i for i in range(R) if i not in none]
        got.append([t.cpu() for t in (dgu.codes.view(torch.uint8), dgu.scales, dgu.codes_t.view(torch.uint8), dgu.scales_t,
                                      h.codes_t.view(torch.uint8), h.scales_t, dw[keep])])
        assert (got[-1][0][none] == 0).all()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# ------------------------------------------------------------------------------------ the layer

LAYERS = [dict(T=1, d=256, f=128, E=8, k=2, score="softmax"), dict(T=300, d=384, f=256, E=16, k=4, score="sigmoid"),
          dict(T=129, d=128, f=384, E=5, k=5, score="softmax", f_shared=256), dict(T=0, d=128, f=128, E=4, k=2, score="softmax"),
          dict(T=700, d=256, f=128, E=300, k=8, score="softmax")]


@pytest.mark.parametrize("c", LAYERS, ids=lambda c: f"T{c['T']}E{c['E']}")
def test_layer(c):
    """Forward and backward, each step against float64 from what the step before left on the GPU."""
    from dropless_mixture_experts_warp_gb300 import layer
    c = dict(c)
    T, d, f, E, k, fs = c["T"], c["d"], c["f"], c["E"], c["k"], c.get("f_shared", 0)
    rng = np.random.default_rng(T + E)
    x, dy = bf16(rng, T, d).cuda(), bf16(rng, T, d).cuda()
    logits = torch.from_numpy((rng.standard_normal((T, E)) + rng.standard_normal(E)).astype(np.float32)).cuda()
    w = {"gu": bf16(rng, E, 2 * f, d, scale=d ** -0.5).cuda(), "d": bf16(rng, E, d, f, scale=f ** -0.5).cuda()}
    sh = {}
    if fs:
        sh = {"w_gu_s": bf16(rng, 2 * fs, d, scale=d ** -0.5).cuda(), "w_d_s": bf16(rng, d, fs, scale=fs ** -0.5).cuda()}
    b = layer.allocate(layer.dims_of(T, d, f, E, k, f_shared=fs, score=c["score"], prec="fp8-block"))
    layer.forward(b, x, logits, w["gu"], w["d"], **sh)
    fwd_h = b.q.h.codes.clone(), b.q.h.scales.clone()
    layer.backward(b, dy, logits, w["gu"], w["d"], x=x, **sh)
    layer.check(b)
    off = b.row_offsets.cpu().tolist()
    n = off[-1]
    idx = b.topk_idx.cpu().numpy()
    assert b.split_sizes.sum() == T * k
    tok = b.row_to_token[:n].cpu().numpy()
    wr = b.w_rows[:n].double().cpu().numpy()

    def routed(a):
        return np.where(tok[:, None] >= 0, a.float().cpu().numpy()[np.maximum(tok, 0)], 0.0) if T else np.zeros((0, d), np.float32)

    for q, src in ((b.q.x, x), (b.q.dy, dy)):
        if n:
            cc, ss = ob.quantize_rows(routed(src))
            same_codes(q.codes[:n], cc)
            assert np.array_equal(q.scales[:, :n].cpu().numpy(), ss)
            cc, ss = ob.quantize_columns(routed(src))
            same_codes(q.codes_t[:, :n].contiguous(), cc)
            assert np.array_equal(q.scales_t[: n // 128].cpu().numpy(), ss)
    vw = {n_: ob.weights_values(w_.codes.cpu(), w_.scales.cpu().numpy()) for n_, w_ in (("gu", b.q.gu), ("d", b.q.down))}
    qc, qs = ob.quantize_weights(w["gu"].float().cpu().numpy())
    same_codes(b.q.gu.codes, qc)

    def val(r, codes=None, scales=None):
        return ob.rows_values((r.codes if codes is None else codes)[:n].cpu(), (r.scales if scales is None else scales)[:, :n].cpu().numpy())

    def cols(r):
        return ob.rows_values(r.codes_t[:, :n].cpu(), r.scales_t[: n // 128].cpu().numpy()).T

    ref, mag = ob.product(val(b.q.x), vw["gu"], off)
    close(b.gu[:n], ref, mag, d)
    gu = b.gu[:n].double().cpu().numpy()
    hr = ob.swiglu(gu[:, :f], gu[:, f:], wr)
    if n:
        stands_for(fwd_h[0][:n], fwd_h[1][:, :n], hr)
        stands_for(b.q.h.codes_t[:, :n], b.q.h.scales_t[: n // 128], hr.T)
    ref, mag = ob.product(val(b.q.h, *fwd_h), vw["d"], off)
    close(b.y_rows[:n], ref, mag, f)
    rows_of = b.token_to_row.cpu().numpy()
    yr = b.y_rows.float().cpu().numpy()
    y = yr[rows_of].astype(np.float64).sum(1) if T else np.zeros((0, d))
    extra = b.y_s.double().cpu().numpy() if fs else 0.0
    close(b.y, y + extra, np.abs(y) + np.abs(extra) + np.abs(yr[rows_of]).sum(1) if T else y, k + 1)
    # backward
    ref, mag = ob.product(val(b.q.dy), vw["d"].transpose(0, 2, 1), off)
    close(b.q.dh[:n], ref, mag, d)
    dh = b.q.dh[:n].double().cpu().numpy()
    dG, dU, dws = ob.swiglu_bwd(gu[:, :f], gu[:, f:], wr, dh)
    if n:
        stands_for(b.q.dgu.codes[:n], b.q.dgu.scales[:, :n], np.concatenate([dG, dU], 1), gradient_terms(gu[:, :f], gu[:, f:], wr, dh))
        assert np.allclose(b.dw_rows[:n].cpu().numpy(), dws, rtol=0, atol=(f + 64) * ob.U32 * 50)
    ref, mag = ob.product(val(b.q.dgu), vw["gu"].transpose(0, 2, 1), off)
    close(b.dxp[:n], ref, mag, 2 * f)
    for got, a, bb in ((b.dw_d, b.q.dy, b.q.h), (b.dw_gu, b.q.dgu, b.q.x)):
        ref, mag = ob.weight_grad(cols(a), cols(bb), off)
        close(got, ref, mag, max(128, max(np.diff(off))))
    if fs and T:
        q = b.q_s
        cc, ss = ob.quantize_rows(x.float().cpu().numpy())
        same_codes(q.x.codes, cc)
        gs = b.gu_s.double().cpu().numpy()
        ref, mag = ob.product(ob.rows_values(cc, ss), ob.weights_values(q.gu.codes.cpu(), q.gu.scales.cpu().numpy()))
        close(b.gu_s, ref, mag, d)
        ref, mag = ob.product(ob.rows_values(q.dgu.codes.cpu(), q.dgu.scales.cpu().numpy()),
                              ob.weights_values(q.gu.codes.cpu(), q.gu.scales.cpu().numpy()).transpose(0, 2, 1))
        close(b.dx_s, ref, mag, 2 * fs)
        ref, mag = ob.weight_grad(ob.rows_values(q.dgu.codes_t.cpu(), q.dgu.scales_t.cpu().numpy()).T,
                                  ob.rows_values(q.x.codes_t.cpu(), q.x.scales_t.cpu().numpy()).T)
        close(b.dw_gu_s, ref[0], mag[0], T)
        stands_for(q.h.codes_t, q.h.scales_t, np.concatenate([ob.swiglu(gs[:, :fs], gs[:, fs:], np.ones(T)), np.zeros((ob.up(T) - T, fs))]).T)
    assert idx.shape == (T, k)


def test_layer_serving_form():
    """train=False with a checkpoint's weights gives the training form's output; backward is refused."""
    from dropless_mixture_experts_warp_gb300 import fp8, layer
    rng = np.random.default_rng(9)
    T, d, f, E, k = 33, 256, 128, 8, 2
    x = bf16(rng, T, d).cuda()
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    w_gu, w_d = bf16(rng, E, 2 * f, d, scale=0.06).cuda(), bf16(rng, E, d, f, scale=0.09).cuda()
    dims = layer.dims_of(T, d, f, E, k, prec="fp8-block")
    full, lean = layer.allocate(dims), layer.allocate(dims, train=False)
    y = layer.forward(full, x, logits, w_gu, w_d).clone()
    with pytest.raises(ValueError):
        layer.forward(lean, x, logits, None, None, weights_cached=True)
    layer.use_weights(lean, fp8.weights_of(full.q.gu.codes, full.q.gu.scales), fp8.weights_of(full.q.down.codes, full.q.down.scales))
    assert torch.equal(layer.forward(lean, x, logits, None, None, weights_cached=True), y)
    with pytest.raises(ValueError):
        layer.backward(lean, x, logits, None, None)


def test_given_weights_are_not_written():
    """quantize_weights() after use_weights() takes weights of its own."""
    from dropless_mixture_experts_warp_gb300 import fp8, layer
    rng = np.random.default_rng(10)
    T, d, f, E, k = 9, 128, 128, 4, 2
    x, logits = bf16(rng, T, d).cuda(), torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    first, second = ([bf16(rng, E, 2 * f, d, scale=0.06).cuda(), bf16(rng, E, d, f, scale=0.09).cuda()] for _ in range(2))
    given = [fp8.quantize_weights(fp8.allocate_weights(*w.shape), w) for w in first]
    kept = [(w.codes.clone().view(torch.uint8), w.scales.clone()) for w in given]
    dims = layer.dims_of(T, d, f, E, k, prec="fp8-block")
    b, other = layer.allocate(dims), layer.allocate(dims)
    layer.use_weights(b, *given)
    with pytest.raises(ValueError):
        layer.forward(b, x, logits, None, None)
    y = layer.forward(b, x, logits, *second)
    assert torch.equal(y, layer.forward(other, x, logits, *second))
    layer.backward(b, x, logits, *second)
    layer.check(b)
    for w, (codes, scales) in zip(given, kept):
        assert torch.equal(w.codes.view(torch.uint8), codes) and torch.equal(w.scales, scales)
