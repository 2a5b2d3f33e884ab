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
                                   (300, 2064, 1456), (1237, 640, 144)])
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
