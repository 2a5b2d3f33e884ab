"""The 8-bit forms that test_gpu_fp8.py does not reach: h's codes from the two SwiGLUs, CTAs of a split product without
blocks, the layer with group-limited routing."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("weighted", [False, True])
def test_h_of_the_gradient_is_the_forward_h(weighted):
    """Where a tile's rows and columns have one scale (its diagonal holds its largest value), both forms of h hold the same
    codes: the gradient quantises the numbers that the forward did, to the last bit."""
    from dropless_mixture_experts_warp_gb300 import binding as B, fp8
    R, f = 8192, 1024
    g = torch.Generator("cuda").manual_seed(11)
    gu = torch.randn(R, 2 * f, device="cuda", generator=g).bfloat16() * 1.5
    at = torch.arange(R, device="cuda")
    diag = at[:, None] % 128 + 128 * torch.arange(f // 128, device="cuda")     # of every tile of 128 columns
    gu[at[:, None], diag], gu[at[:, None], f + diag] = 8.0, 16.0
    w = torch.rand(R, device="cuda", generator=g) * 0.5 + 0.5 if weighted else None
    if weighted:
        w.view(-1, 128)[:, :] = w[::128, None]                                 # one weight for a tile's rows
    h, ht, dgu = fp8.allocate_rows(R, f), fp8.allocate_rows(R, f, both=True), fp8.allocate_rows(R, 2 * f, both=True)
    B.moe_fp8_swiglu(gu, w, R, f, None, h.codes, h.scales)
    dh = torch.randn(R, f, device="cuda", generator=g).bfloat16()
    B.moe_fp8_swiglu_bwd(gu, dh, w, R, f, None, dgu.codes, dgu.scales, dgu.codes_t, dgu.scales_t, ht.codes_t, ht.scales_t, None, None)
    rows = h.scales.view(f // 128, R // 128, 128)
    assert torch.equal(rows, ht.scales_t.view(R // 128, f // 128, 128).transpose(0, 1))
    assert torch.equal(rows, rows[:, :, :1].expand_as(rows))
    different = h.codes.view(torch.uint8) != ht.codes_t.view(torch.uint8).t()
    assert not different.any(), int(different.sum())


@pytest.mark.parametrize("count", [-1, -128, -300, -(1 << 31), 0])
def test_counts_below_zero_are_no_rows(count):
    """A count of rows that is negative counts as none: every buffer stays as it was."""
    from dropless_mixture_experts_warp_gb300 import binding as B, fp8
    R, f = 300, 256
    n = torch.tensor([count], dtype=torch.int32).cuda()
    x, dh = torch.randn(R, 2 * f, device="cuda").bfloat16(), torch.randn(R, f, device="cuda").bfloat16()
    a, d, h = fp8.allocate_rows(R, 2 * f, both=True), fp8.allocate_rows(R, 2 * f, both=True), fp8.allocate_rows(R, f, both=True)
    dw, part, w = torch.full((R,), 7.0, device="cuda"), torch.full((R, f // 128), 7.0, device="cuda"), torch.ones(R, device="cuda")
    codes = [t.view(torch.uint8).fill_(0x11) for r in (a, d, h) for t in (r.codes, r.codes_t)]
    scales = [t.fill_(7.0) for r in (a, d, h) for t in (r.scales, r.scales_t)]
    B.moe_fp8_quantize(x, R, 2 * f, None, n, a.codes, a.scales, a.codes_t, a.scales_t)
    B.moe_fp8_quantize(x, R, 2 * f, None, n, a.codes, a.scales, None, None)
    B.moe_fp8_swiglu(x, w, R, f, n, h.codes, h.scales)
    B.moe_fp8_swiglu_bwd(x, dh, w, R, f, n, d.codes, d.scales, d.codes_t, d.scales_t, h.codes_t, h.scales_t, dw, part)
    assert all((t == 0x11).all() for t in codes) and all((t == 7.0).all() for t in scales + [dw, part])


@pytest.mark.parametrize("R,K", [(1, 4224), (5, 4352), (128, 4480), (3, 4608), (7, 4256), (2, 2176), (130, 5376)])
@pytest.mark.parametrize("transposed", [False, True])
def test_split_products_of_odd_numbers_of_blocks(R, K, transposed):
    """33 to 36 and other numbers of blocks over up to eight CTAs a tile: shares differ, the last may be empty."""
    from dropless_mixture_experts_warp_gb300 import fp8
    from test_gpu_fp8 import close, cuda, rows, weights
    from oracle import blocks as ob
    N = 272
    rng = np.random.default_rng(R + K)
    a = rows(rng, R, K)
    w = weights(rng, 1, K, N) if transposed else weights(rng, 1, N, K)
    more = {"codes_t": cuda(w[0].transpose(1, 2).contiguous())} if transposed else {}
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    x = fp8.rows_of(*map(cuda, a[:2]))
    fp8.matmul(x, fp8.weights_of(*map(cuda, w), **more), out, transposed=transposed)
    fp8.check(x)
    v = ob.weights_values(w[0], w[1])
    ref, mag = ob.product(ob.rows_values(*a[:2]), v.transpose(0, 2, 1) if transposed else v)
    close(out, ref, mag, K)


@pytest.mark.parametrize("T,E,k,n_group,topk_group,fs", [(300, 16, 4, 4, 2, 256), (5, 256, 8, 8, 4, 128), (77, 32, 6, 8, 3, 0)])
def test_layer_with_group_limited_routing(T, E, k, n_group, topk_group, fs):
    """A DeepSeek-V3 router (groups, bias, routed scale) before the layer in this form, forward and backward: the choices
    are the bf16 layer's, and each step after them is right from what the step before left on the GPU."""
    from dropless_mixture_experts_warp_gb300 import fp8, layer
    from test_gpu_fp8 import bf16, close
    from oracle import blocks as ob
    d, f, scale = 256, 128, 2.5
    rng = np.random.default_rng(T + E)
    x, dy = bf16(rng, T, d).cuda(), bf16(rng, T, d).cuda()
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    bias = torch.from_numpy((rng.standard_normal(E) * 0.2).astype(np.float32)).cuda()
    gr = {"n_group": n_group, "topk_group": topk_group, "bias": bias, "routed_scale": scale}
    w_gu, w_d = bf16(rng, E, 2 * f, d, scale=d ** -0.5).cuda(), bf16(rng, E, d, f, scale=f ** -0.5).cuda()
    sh = {"w_gu_s": bf16(rng, 2 * fs, d, scale=d ** -0.5).cuda(), "w_d_s": bf16(rng, d, fs, scale=fs ** -0.5).cuda()} if fs else {}
    make = lambda prec, **kw: layer.allocate(layer.dims_of(T, d, f, E, k, f_shared=fs, score="sigmoid", prec=prec), **kw)  # noqa: E731
    b, plain, lean = make("fp8-block"), make("bf16"), make("fp8-block", train=False)
    layer.forward(b, x, logits, w_gu, w_d, grouped=gr, **sh)
    layer.forward(plain, x, logits, w_gu, w_d, grouped=gr, **sh)
    assert torch.equal(b.topk_idx, plain.topk_idx) and torch.equal(b.topk_w, plain.topk_w) and torch.equal(b.row_offsets, plain.row_offsets)
    assert torch.allclose(b.topk_w.sum(1), torch.full((T,), scale, device="cuda"), rtol=1e-5)
    y = b.y.clone()
    shared = (b.q_s.gu, b.q_s.down) if fs else ()
    layer.use_weights(lean, b.q.gu, b.q.down, *shared)
    assert torch.equal(layer.forward(lean, x, logits, None, None, grouped=gr, weights_cached=True), y)
    rows = b.token_to_row.cpu().numpy()
    yr = b.y_rows.double().cpu().numpy()[rows]
    extra = b.y_s.double().cpu().numpy() if fs else 0.0
    close(y, yr.sum(1) + extra, np.abs(yr).sum(1) + np.abs(extra), k + 1)
    off = b.row_offsets.tolist()
    n = off[-1]
    hv = ob.rows_values(b.q.h.codes[:n].cpu(), b.q.h.scales[:, :n].cpu().numpy())
    ref, mag = ob.product(hv, ob.weights_values(b.q.down.codes.cpu(), b.q.down.scales.cpu().numpy()), off)
    close(b.y_rows[:n], ref, mag, f)
    layer.backward(b, dy, logits, w_gu, w_d, x=x, grouped=gr, **sh)
    layer.check(b)
    dxp = b.dxp.double().cpu().numpy()[rows]
    extra = b.dx_s.double().cpu().numpy() if fs else 0.0
    close(b.dx, dxp.sum(1) + extra, np.abs(dxp).sum(1) + np.abs(extra), k + 1)
    # w_j = scale s_j / sum of the chosen s, s = sigmoid(logit): d logit_j = scale s_j (1 - s_j) (dw_j - sum_i dw_i s_i / S) / S
    idx = b.topk_idx.long().cpu().numpy()
    s = ob.sigmoid(np.take_along_axis(logits.double().cpu().numpy(), idx, 1))
    S = s.sum(1, keepdims=True)
    dw = b.dw_rows.double().cpu().numpy()[rows]
    slope = scale * s * (1 - s) / S
    ref, mag = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(ref, idx, slope * (dw - (dw * s).sum(1, keepdims=True) / S), 1)
    np.put_along_axis(mag, idx, slope * (np.abs(dw) + (np.abs(dw) * s).sum(1, keepdims=True) / S), 1)
    # fp32: exponentials good to 2^-20, k terms
    assert np.all(np.abs(b.d_logits.double().cpu().numpy() - ref) <= (2.0 ** -18 + (k + 8) * ob.U32) * mag)
