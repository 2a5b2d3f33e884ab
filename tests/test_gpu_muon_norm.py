"""The norm that Muon's matrices are divided by, over the range of fp32: gradients and momenta of any size, idle experts.

Bounds: those of test_gpu_muon.py (its `near`), whose derivation stands there; and equal bits where inputs differ by a
power of two, which no rounding of the kernels sees.
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from oracle import blocks as ob
from test_gpu_muon import matrices, near

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("products", ["fp32", "fp16"])
SHAPES = [(96, 160), (40, 7), (300, 200), (129, 257)]      # the first two in one block, the others through the workspace


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def orthogonal(x, products):
    from dropless_mixture_experts_warp_gb300 import muon
    w = muon.workspace([x.shape], products=products)
    o = torch.empty(x.shape, device="cuda")
    muon.orthogonalize([x.cuda()], [o], w)
    muon.check(w)
    return o


@both
@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_any_scale(m, n, kind, products):
    """x times a power of two has x's orthogonal factor, bit for bit, also where squares of its elements are below fp32."""
    x = matrices(np.random.default_rng(m), 1, m, n, kind, scale=1.0)
    want = orthogonal(x, products)
    near(want[0], x[0].double().numpy(), torch.float32)
    for e in (30, -20, -45, -55, -62, -66, -70, -75, -90):
        y = x * 2.0 ** e
        assert torch.equal(y.double(), x.double() * 2.0 ** e)      # nothing of x is lost
        assert torch.equal(orthogonal(y, products), want), e


@both
@pytest.mark.parametrize("m,n", SHAPES)
def test_subnormal_elements(m, n, products):
    x = matrices(np.random.default_rng(n), 1, m, n, torch.float32, scale=2.0 ** -136)
    assert 0 < x.abs().max() < 2.0 ** -126
    near(orthogonal(x, products)[0], x[0].double().numpy(), torch.float32)


@both
@pytest.mark.parametrize("m,n", SHAPES)
def test_matrices_of_different_sizes_together(m, n, products):
    """Each matrix of a batch by its own norm."""
    x = matrices(np.random.default_rng(3), 5, m, n, torch.float32, scale=1.0)
    for i, e in enumerate((0, -70, -100, 20, -60)):
        x[i] *= 2.0 ** e
    x[2] = 0.0
    o = orthogonal(x, products)
    assert (o[2] == 0).all()
    for i in (0, 1, 3, 4):
        near(o[i], x[i].double().numpy(), torch.float32)


@both
@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("rank", [1, 4, None])
def test_idle_expert(m, n, rank, products):
    """An expert without tokens has gradients of zeros: its momentum shrinks by 0.95 a step until it is gone, and its
    weights stay finite."""
    from dropless_mixture_experts_warp_gb300 import muon
    rng = np.random.default_rng(5)
    if rank is None:
        mom = matrices(rng, 2, m, n, torch.float32)
    else:
        mom = torch.from_numpy(1e-4 * rng.standard_normal((2, m, rank)) @ rng.standard_normal((2, rank, n))).float()
    w = torch.from_numpy(rng.standard_normal((2, m, n)).astype(np.float32) * 0.02).cuda()
    low = w.bfloat16()
    p = muon.plan([w], [torch.zeros(2, m, n, device="cuda")], copies=[low], m=[mom.cuda()], products=products)
    for t in range(1, 2101):
        muon.step(p, lr=1e-3)
        if t % 25 == 0:
            assert torch.isfinite(w).all() and torch.isfinite(p.m[0]).all(), t
    muon.check(p)
    assert torch.isfinite(low).all()


@pytest.mark.parametrize("m,n", SHAPES)
def test_idle_expert_comes_to_rest(m, n):
    """The steps of an expert without tokens fade below eps, as the definition's do."""
    from dropless_mixture_experts_warp_gb300 import muon
    rng = np.random.default_rng(6)
    mom = matrices(rng, 2, m, n, torch.float32)
    w = torch.from_numpy(rng.standard_normal((2, m, n)).astype(np.float32) * 0.02).cuda()
    p = muon.plan([w], [torch.zeros(2, m, n, device="cuda")], m=[mom.cuda()])
    for _ in range(800):
        muon.step(p, lr=1e-3)
    rest = w.clone()
    for _ in range(400):
        muon.step(p, lr=1e-3)
    muon.check(p)
    # |U| started below 0.1 and is below 0.1 x 0.95^800 = 2^-62 after 800 steps, 2^-38 of eps; five steps make a
    # singular value at most 3.4445^5 < 2^9 times as large, so an update's norm is below lr rms sqrt(max side)
    # 2^-29, and all that follow add up to 20 of them, for each of two matrices; adding them rounds w below half a step
    assert mom.norm() < 0.1
    size = 1e-3 * 0.2 * np.sqrt(max(m, n))
    assert (w - rest).norm().item() <= 2 * 20 * size * 2.0 ** -29


@both
@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("times", [0.0, 0.3, 1.0, 5.0, 1e4])
def test_floor(m, n, times, products):
    """X_0 = U / max(|U|, eps), against float64."""
    from dropless_mixture_experts_warp_gb300 import muon
    rng = np.random.default_rng(m + 1)
    g = matrices(rng, 1, m, n, torch.float32)[0]
    w0 = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32) * 0.02)
    eps = times * g.double().norm().item()
    w = w0.cuda()
    p = muon.plan([w], [g.cuda()], products=products)
    lr, rms = 2e-2, 0.2
    muon.step(p, lr=lr, momentum=0.0, rms=rms, nesterov=False, eps=eps)
    muon.check(p)
    u = g.double().numpy()
    ref, _, o = ob.muon_step(w0.double().numpy(), np.zeros((m, n)), u, lr, 0.0, 0.0, rms, False, eps=eps)
    low = ob.newton_schulz_rounded(u, eps=eps)
    e = np.linalg.norm((low.T if m > n else low) - o)
    size = lr * rms * np.sqrt(max(m, n))
    off = np.linalg.norm(w.double().cpu().numpy() - ref)
    # as in test_gpu_muon.py's test_step, and fp16's smallest steps, 2^-25 of an element of X_0 in its second
    # part, which five steps make at most 2^9 times as large: they count where X_0 is small
    fine = 2.0 ** -16 * np.sqrt(m * n)
    assert off <= size * (1.5 * e + 2.0 ** -11 * np.linalg.norm(o) + fine) + 4 * ob.U32 * np.linalg.norm(np.abs(ref) + size * np.abs(o))
