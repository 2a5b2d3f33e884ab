"""Muon's way through the workspace (matrices past 128 x 256): several tensors of a shape in a launch, batches that a
chunk ends in, tall and odd ones with momenta and weights, scales and skips from the device, other steps than the default.

Bounds against float64: as in test_gpu_muon.py, 1.5 times what the same roundings cost in float64 and a rounding of the
result; and beside it what the documentation states for any matrix, by its shorter side (LIMIT), so that the scheme's
own error is held too.
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from oracle import blocks as ob
from test_gpu_muon import HALF, matrices, run_step

pytestmark = pytest.mark.gpu
LR, MU, RMS = 2e-3, 0.95, 0.2
SHAPES = [(3, 200, 300), (300, 200), (2, 129, 257), (200, 300), (257, 129), (2, 2, 300, 200), (131, 72), (129, 257)]
# relative to the factor's norm: seen over 1042 matrices of both kinds, 1 to 600 rows, aspect up to 12: 7.7e-3 below
# 16, 3.0e-3 below 128, 1.2e-3 from there on
LIMIT = lambda side: 1e-2 if side < 16 else 4e-3 if side < 128 else 1.5e-3  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def flat(t, s):
    return t.double().cpu().numpy().reshape(-1, *s[-2:])


def check_step(p, start, gs, low, shapes, nesterov=True, grad_scale=1.0, lr=LR, decay=None, coefficients=ob.COEFFICIENTS):
    """p after one step from start = (w, m), with grad_scale's gradients, against float64."""
    for i, s in enumerate(shapes):
        m, n = s[-2:]
        wd = 0.1 * (i + 1) if decay is None else decay
        for w, mm, g, nw, nm in zip(flat(start[0][i], s), flat(start[1][i], s), flat(gs[i], s), flat(p.weights[i], s), flat(p.m[i], s)):
            g = g * float(np.float32(grad_scale))
            ref, mref, o = ob.muon_step(w, mm, g, lr, MU, wd, RMS, nesterov, coefficients)
            assert np.all(np.abs(nm - mref) <= 4 * ob.U32 * (np.abs(MU * mm) + np.abs(g))), s      # a product, one fma
            u = g + MU * mref if nesterov else mref
            rounded = ob.newton_schulz_rounded(u, coefficients)
            e = np.linalg.norm((rounded.T if m > n else rounded) - o)
            size = lr * RMS * np.sqrt(max(m, n))
            fp32 = 4 * ob.U32 * np.linalg.norm(np.abs(w) + size * np.abs(o))
            off = np.linalg.norm(nw - ref)
            assert off <= size * (1.5 * e + 2.0 ** -11 * np.linalg.norm(o)) + fp32, s
            if coefficients == ob.COEFFICIENTS:
                assert off <= size * (LIMIT(min(m, n)) + 2.0 ** -11) * np.linalg.norm(o) + fp32, s
        if low[i] is not None:
            assert torch.equal(low[i], p.weights[i].bfloat16())


@pytest.mark.parametrize("kind,nesterov,copies", [(torch.bfloat16, True, True), (torch.float32, False, False), (torch.float32, True, True)])
def test_step(kind, nesterov, copies):
    p, start, gs, low = run_step(SHAPES, kind, copies, nesterov, steps=1)
    check_step(p, start, gs, low, SHAPES, nesterov)


def test_chunks():
    """Workspaces of one, two and five matrices and of all give the same bits: batches that a chunk ends in, a chunk that
    holds the end of one tensor and the start of the next, more tensors of a shape than a launch takes."""
    from dropless_mixture_experts_warp_gb300 import binding as B, muon
    shapes = [(3, 200, 300), (200, 300), (5, 200, 300), (300, 200), (4, 300, 200), (2, 129, 257)] + [(129, 200)] * 35 + [(2, 129, 200)]
    one = max(muon.workspace([s], limit=1).workspace.numel() for s in shapes)
    big = run_step(shapes)[0]
    check_step(*run_step(shapes, steps=1), shapes)
    for matrices_at_once in (1, 2, 5):
        other = run_step(shapes, workspace=matrices_at_once * one)[0]
        assert matrices_at_once * one - one < other.workspace.numel() <= matrices_at_once * one < big.workspace.numel()
        for a, b, c, d in zip(big.weights + big.m, other.weights + other.m, big.copies, other.copies):
            assert torch.equal(a, b) and torch.equal(c, d)
    assert B.MUON_MAX_STEPS >= 6


@pytest.mark.parametrize("shapes", [[(64, 96), (2, 33, 40)], [(2, 300, 200), (129, 257), (200, 300)]])
def test_scales_from_the_device(shapes):
    from dropless_mixture_experts_warp_gb300 import optim
    c = optim.Control()
    for grad_scale, lr_scale in ((0.37, 1.0), (1.0, 0.5), (512.0, 0.25)):
        c.grad_scale.fill_(grad_scale)
        c.lr_scale.fill_(lr_scale)
        for nesterov in (True, False):
            p, start, gs, low = run_step(shapes, nesterov=nesterov, control=c, steps=1)
            check_step(p, start, gs, low, shapes, nesterov, grad_scale, LR * lr_scale)


@pytest.mark.parametrize("shapes", [[(64, 96), (2, 33, 40)], [(2, 300, 200), (129, 257), (200, 300)]])
def test_skip_leaves_everything(shapes):
    """Whatever the gradients hold."""
    from dropless_mixture_experts_warp_gb300 import muon, optim
    p, _, gs, low = run_step(shapes, steps=1)
    for g, fill in zip(gs, (float("nan"), float("inf"), -float("inf"))):
        g[..., 1:3, 2:4] = fill
    before = [t.clone() for t in p.weights + p.m + low]
    c = optim.Control()
    c.skip.fill_(1)
    muon.step(p, lr=LR, control=c)
    muon.check(p)
    assert all(torch.equal(a, b) for a, b in zip(p.weights + p.m + low, before))


@pytest.mark.parametrize("m,n", [(40, 100), (96, 160), (300, 200), (129, 257), (256, 700)])
@pytest.mark.parametrize("coefficients", [[(1.5, -0.5, 0.0)], [(3.4445, -4.7750, 2.0315)] * 2, [(1.5, -0.5, 0.0)] * 2 + [(3.4445, -4.7750, 2.0315)] * 4,
                                          [(1.875, -1.25, 0.375)] * 16])
def test_other_steps(m, n, coefficients):
    from dropless_mixture_experts_warp_gb300 import muon
    x = matrices(np.random.default_rng(m * n), 2, m, n, torch.float32)
    w = muon.workspace([x.shape], coefficients=coefficients)
    o = torch.empty(x.shape, device="cuda")
    muon.orthogonalize([x.cuda()], [o], w)
    muon.check(w)
    for i in range(2):
        v = x[i].double().numpy()
        ref, low = ob.newton_schulz(v, coefficients), ob.newton_schulz_rounded(v, coefficients)
        e = np.linalg.norm((low.T if m > n else low) - ref)
        assert np.linalg.norm(o[i].double().cpu().numpy() - ref) <= 1.5 * e + (HALF[torch.float32] + 2.0 ** -20) * np.linalg.norm(ref)


@pytest.mark.parametrize("m,n", [(1, 1), (7, 40), (16, 16), (16, 40), (31, 300), (72, 131), (128, 128), (129, 257), (200, 2000), (640, 384), (512, 512)])
@pytest.mark.parametrize("gaussian", [True, False])
def test_how_far_the_factor_is(m, n, gaussian):
    """The error that the documentation states, whatever the kernels' own scheme of roundings costs."""
    from dropless_mixture_experts_warp_gb300 import muon
    rng = np.random.default_rng(m + 7 * n)
    x = torch.from_numpy(rng.standard_normal((3, m, n)).astype(np.float32)) if gaussian else matrices(rng, 3, m, n, torch.float32)
    w = muon.workspace([x.shape])
    o = torch.empty(x.shape, device="cuda")
    muon.orthogonalize([x.cuda()], [o], w)
    for i in range(3):
        ref = ob.newton_schulz(x[i].double().numpy())
        off = np.linalg.norm(o[i].double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert off <= LIMIT(min(m, n)), off


def test_in_place_and_shared_inputs():
    """An output that is its own input, in one block, through the workspace and in chunks."""
    from dropless_mixture_experts_warp_gb300 import muon
    for s in [(5, 64, 96), (5, 300, 200)]:
        x = matrices(np.random.default_rng(2), *s, torch.float32).cuda()
        want, ws = torch.empty_like(x), muon.workspace([s, s], limit=1)
        again = torch.empty_like(x)
        muon.orthogonalize([x, x], [want, again], ws)
        y = x.clone()
        muon.orthogonalize([y, x], [y, again], ws)
        assert torch.equal(y, want) and torch.equal(again, want)
