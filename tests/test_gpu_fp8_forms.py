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
