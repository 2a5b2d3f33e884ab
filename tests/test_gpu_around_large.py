"""The operators around the layer on tensors whose element offsets pass 32 bits (GPU)."""
import numpy as np
import pytest
import torch

from oracle import around as oa
from tests.around_util import check
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
PAST = (1 << 32) + 3 * 8192     # elements: the last rows lie past 2^32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()
    if torch.cuda.get_device_properties(0).total_memory < 100e9:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def test_norms():
    from dropless_mixture_experts_warp_gb300 import block
    d = 8192
    T = PAST // d
    rows = torch.tensor([0, (1 << 31) // d - 1, (1 << 31) // d, (1 << 32) // d - 1, (1 << 32) // d, T - 1], device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    h, dx = (torch.ones(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (h, dx):
        t[rows] = torch.randn(len(rows), d, device="cuda", generator=g).bfloat16()
    w = torch.randn(d, device="cuda", generator=g)
    dims = block.dims_of(T, d)
    # the entry points themselves: allocate() would hold every call's outputs at once
    from dropless_mixture_experts_warp_gb300 import binding as B
    out, dw = torch.empty_like(h), torch.empty(d, device="cuda")
    ws = torch.empty(B.moe_norm_workspace_size(dims), dtype=torch.uint8, device="cuda")
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    B.moe_norm_fwd(dims, h, w, out)
    x = oa.norm_fwd(f64(h[rows]), f64(w), 1e-6)
    check("x", out[rows], (x, abs(x)), "bf16", 128)
    B.moe_norm_bwd(dims, dx, h, w, None, out, dw, ws)
    check("dh", out[rows], oa.norm_bwd(f64(dx[rows]), f64(h[rows]), f64(w), 1e-6)["dh"], "bf16", 128)
    x_next = torch.empty_like(h)
    B.moe_merge_fwd(dims, h, dx, w, None, w, out, x_next)
    ref = oa.merge_fwd(f64(h[rows]), f64(dx[rows]), f64(w), None, f64(w), eps=1e-6)
    check("h_out", out[rows], ref["h_out"], "bf16", 128)
    check("x_next", x_next[rows], ref["x"], "bf16", 256)


def test_balance():
    from dropless_mixture_experts_warp_gb300 import balance
    E, k = 1024, 1
    T = PAST // E // 2          # 2^31 logits, 2^33 bytes
    rows = [0, (1 << 20) - 1, T // 2, T - 2, T - 1]
    l = torch.zeros(T, E, device="cuda")
    l[rows] = torch.randn(len(rows), E, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    idx[-1] = 7
    b = balance.allocate(T, E, k)
    balance.forward(b, l, idx, z_coef=1.0)
    balance.check(b)
    assert int(b.counts[0, 0]) == T - 1 and int(b.counts[0, 7]) == 1
    d = torch.zeros(T, E, device="cuda")
    balance.backward(b, l, d, z_coef=1.0)
    counts, n = b.counts.cpu().numpy().astype(np.int64), np.array([T])
    sub = l[rows].double().cpu().numpy()
    # the formula of a row, with the whole batch's counts and number of tokens
    p = oa.probabilities(sub, "softmax")
    f = E * counts[0] / T
    m = (f * p).sum(axis=1, keepdims=True)
    lse = oa.logsumexp(sub)[:, None]
    want = p * (f - m) / T + 2 / T * lse * p
    check("d_logits", d[rows], (want, p * (f + m) / T + 2 / T * abs(lse) * p), "fp32", 256)


def test_adamw():
    from dropless_mixture_experts_warp_gb300 import optim
    n = (1 << 32) + 5000
    w, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5000, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) * 1e-2
    first = 1 << 32             # a block of 128 starts here
    g[first:] = tail
    p = optim.plan([w], [g], bits=8)
    optim.step(p, lr=1e-2, step=1, seed=9)
    g64 = g[first:].double().cpu().numpy()
    m = 0.1 * g64
    ref = oa.block_scales(m)
    want, margin = oa.encode(m, ref, oa.adamw_draws(9, 1, 0, 5000, first)[0], 127, 2)
    got = p.m[0][first:].cpu().numpy().astype(np.int64)
    low = np.maximum(abs(want) - 1, 0)
    near = margin <= 24 * oa.U32 * np.repeat(ref, 128)[:5000] / np.repeat(ref, 128)[:5000] / ((2 * low + 1) / 16129)
    assert np.array_equal(got[~near], want[~near]) and near.mean() < 0.05
    assert torch.count_nonzero(w[:first]) == 0
    # the first step: m / (1 - beta1) = g, v / (1 - beta2) = g^2
    want_w = -1e-2 * g64 / (abs(g64) + 1e-8)
    check("w", w[first:], (want_w, abs(want_w)), "fp32", 32)
