"""Muon's way through the workspace (matrices past 128 x 256): several tensors of a shape in a launch, batches that a
chunk ends in, tall and odd ones with momenta and weights, scales and skips from the device, other steps than the default.

Bounds against float64: as in test_gpu_muon.py, 1.5 times what the same roundings cost in float64 and a rounding of the
result; with operands in two parts also what their fp32 sums may lose (newton_schulz_split).  Beside it what the
documentation states for any matrix (LIMIT), so that the scheme's own error is held too.
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from oracle import blocks as ob
from test_gpu_muon import HALF, matrices

pytestmark = pytest.mark.gpu
LR, MU, RMS = 2e-3, 0.95, 0.2
SHAPES = [(3, 200, 300), (300, 200), (2, 129, 257), (200, 300), (257, 129), (2, 2, 300, 200), (131, 72), (129, 257)]
PRODUCTS = ["fp32", "fp16"]


def limit(m, n, products):
    """Relative to the factor's norm.  fp16, seen over 1042 matrices of both kinds, 1 to 600 rows, aspect up to 12: 7.7e-3
    below 16 rows, 3.0e-3 below 128, 1.2e-3 from there on.  fp32: operands of 22 bits, five steps of which lose 3e-6
    at 1024; and sums that lose half a unit in the last place, 2^-24, at each of their l / 16 steps where they grow
    evenly, as on A's diagonal: l 2^-28, which a step's |b| + 2 |c| = 9 and those after it make up to 20 times as large."""
    if products == "fp32":
        return 1e-5 + max(m, n) * 20 * 2.0 ** -28
    return 1e-2 if min(m, n) < 16 else 4e-3 if min(m, n) < 128 else 1.5e-3


def cost(u, o, products, coefficients=ob.COEFFICIENTS):
    """What the arithmetic costs of u's factor o, in norm."""
    turn = lambda r: r.T if u.shape[0] > u.shape[1] else r  # noqa: E731
    if products == "fp16":
        return 1.5 * np.linalg.norm(turn(ob.newton_schulz_rounded(u, coefficients)) - o)
    operands = turn(ob.newton_schulz_split(u, coefficients, step=0))
    return 1.5 * np.linalg.norm(operands - o) + np.linalg.norm(turn(ob.newton_schulz_split(u, coefficients)) - operands)


def run_step(shapes, kind=torch.bfloat16, copies=True, nesterov=True, workspace=1 << 30, steps=2, control=None, products="fp32"):
    from dropless_mixture_experts_warp_gb300 import muon
    rng = np.random.default_rng(0)
    ws, gs, ms = [], [], []
    for s in shapes:
        b = int(np.prod(s[:-2]))
        ws.append(torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.02).cuda())
        gs.append(matrices(rng, b, s[-2], s[-1], kind).reshape(s).cuda())
        ms.append(matrices(rng, b, s[-2], s[-1], torch.float32, 5e-4).reshape(s).cuda())
    low = [w.bfloat16() if copies else None for w in ws]
    start = [w.clone() for w in ws], [m.clone() for m in ms]
    p = muon.plan(ws, gs, copies=low, m=ms, weight_decay=[0.1 * (i + 1) for i in range(len(ws))], workspace=workspace, products=products)
    for _ in range(steps):
        muon.step(p, lr=LR, momentum=MU, rms=RMS, nesterov=nesterov, control=control)
    muon.check(p)
    return p, start, gs, low


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def flat(t, s):
    return t.double().cpu().numpy().reshape(-1, *s[-2:])


def check_step(p, start, gs, low, shapes, products, nesterov=True, grad_scale=1.0, lr=LR):
    """p after one step from start = (w, m), with grad_scale's gradients, against float64."""
    for i, s in enumerate(shapes):
        m, n = s[-2:]
        for w, mm, g, nw, nm in zip(flat(start[0][i], s), flat(start[1][i], s), flat(gs[i], s), flat(p.weights[i], s), flat(p.m[i], s)):
            g = g * float(np.float32(grad_scale))
            ref, mref, o = ob.muon_step(w, mm, g, lr, MU, 0.1 * (i + 1), RMS, nesterov)
            assert np.all(np.abs(nm - mref) <= 4 * ob.U32 * (np.abs(MU * mm) + np.abs(g))), s      # a product, one fma
            u = g + MU * mref if nesterov else mref
            result = {"fp16": 2.0 ** -11, "fp32": 2.0 ** -21}[products]         # X's last form
            size = lr * RMS * np.sqrt(max(m, n))
            fp32 = 4 * ob.U32 * np.linalg.norm(np.abs(w) + size * np.abs(o))
            off = np.linalg.norm(nw - ref)
            assert off <= size * (cost(u, o, products) + result * np.linalg.norm(o)) + fp32, s
            assert off <= size * (limit(m, n, products) + result) * np.linalg.norm(o) + fp32, s
        if low[i] is not None:
            assert torch.equal(low[i], p.weights[i].bfloat16())


@pytest.mark.parametrize("products", PRODUCTS)
@pytest.mark.parametrize("kind,nesterov,copies", [(torch.bfloat16, True, True), (torch.float32, False, False), (torch.float32, True, True)])
def test_step(kind, nesterov, copies, products):
    p, start, gs, low = run_step(SHAPES, kind, copies, nesterov, steps=1, products=products)
    check_step(p, start, gs, low, SHAPES, products, nesterov)


@pytest.mark.parametrize("products", PRODUCTS)
def test_chunks(products):
    """Workspaces of one, two and five matrices and of all give the same bits: batches that a chunk ends in, a chunk that
    holds the end of one tensor and the start of the next, more tensors of a shape than a launch takes."""
    from dropless_mixture_experts_warp_gb300 import muon
    shapes = [(3, 200, 300), (200, 300), (5, 200, 300), (300, 200), (4, 300, 200), (2, 129, 257)] + [(129, 200)] * 35 + [(2, 129, 200)]
    one = max(muon.workspace([s], limit=1, products=products).workspace.numel() for s in shapes)
    big = run_step(shapes, products=products)[0]
    check_step(*run_step(shapes, steps=1, products=products), shapes, products)
    for matrices_at_once in (1, 2, 5):
        other = run_step(shapes, workspace=matrices_at_once * one, products=products)[0]
        assert matrices_at_once * one - one < other.workspace.numel() <= matrices_at_once * one < big.workspace.numel()
        for a, b, c, d in zip(big.weights + big.m, other.weights + other.m, big.copies, other.copies):
            assert torch.equal(a, b) and torch.equal(c, d)


@pytest.mark.parametrize("shapes", [[(64, 96), (2, 33, 40)], [(2, 300, 200), (129, 257), (200, 300)]])
@pytest.mark.parametrize("products", PRODUCTS)
def test_scales_from_the_device(shapes, products):
    from dropless_mixture_experts_warp_gb300 import optim
    c = optim.Control()
    for grad_scale, lr_scale in ((0.37, 1.0), (1.0, 0.5), (512.0, 0.25)):
        c.grad_scale.fill_(grad_scale)
        c.lr_scale.fill_(lr_scale)
        for nesterov in (True, False):
            p, start, gs, low = run_step(shapes, nesterov=nesterov, control=c, steps=1, products=products)
            check_step(p, start, gs, low, shapes, products, nesterov, grad_scale, LR * lr_scale)


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
@pytest.mark.parametrize("products", PRODUCTS)
def test_other_steps(m, n, coefficients, products):
    from dropless_mixture_experts_warp_gb300 import muon
    x = matrices(np.random.default_rng(m * n), 2, m, n, torch.float32)
    w = muon.workspace([x.shape], coefficients=coefficients, products=products)
    o = torch.empty(x.shape, device="cuda")
    muon.orthogonalize([x.cuda()], [o], w)
    muon.check(w)
    for i in range(2):
        v = x[i].double().numpy()
        ref = ob.newton_schulz(v, coefficients)
        bound = cost(v, ref, products, coefficients) + (HALF[torch.float32] + 2.0 ** -20) * np.linalg.norm(ref)
        assert np.linalg.norm(o[i].double().cpu().numpy() - ref) <= bound


@pytest.mark.parametrize("m,n", [(1, 1), (7, 40), (16, 16), (16, 40), (31, 300), (72, 131), (128, 128), (129, 257), (200, 2000), (640, 384), (512, 512),
                                 (1024, 1024)])
@pytest.mark.parametrize("gaussian", [True, False])
@pytest.mark.parametrize("products", PRODUCTS)
def test_how_far_the_factor_is(m, n, gaussian, products):
    """The error that the documentation states, whatever the kernels' own scheme of roundings costs."""
    from dropless_mixture_experts_warp_gb300 import muon
    rng = np.random.default_rng(m + 7 * n)
    x = torch.from_numpy(rng.standard_normal((3, m, n)).astype(np.float32)) if gaussian else matrices(rng, 3, m, n, torch.float32)
    w = muon.workspace([x.shape], products=products)
    o = torch.empty(x.shape, device="cuda")
    muon.orthogonalize([x.cuda()], [o], w)
    muon.check(w)
    for i in range(3):
        ref = ob.newton_schulz(x[i].double().numpy())
        off = np.linalg.norm(o[i].double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert off <= limit(m, n, products), off


@pytest.mark.parametrize("products", PRODUCTS)
def test_in_place_and_shared_inputs(products):
    """An output that is its own input, in one block, through the workspace and in chunks."""
    from dropless_mixture_experts_warp_gb300 import muon
    for s in [(5, 64, 96), (5, 300, 200)]:
        x = matrices(np.random.default_rng(2), *s, torch.float32).cuda()
        want, ws = torch.empty_like(x), muon.workspace([s, s], limit=1, products=products)
        again = torch.empty_like(x)
        muon.orthogonalize([x, x], [want, again], ws)
        y = x.clone()
        muon.orthogonalize([y, x], [y, again], ws)
        assert torch.equal(y, want) and torch.equal(again, want)


def test_captured_and_repeated():
    """Both kinds of products in a graph, replayed, give the eager steps' bits, whatever the workspace held before."""
    from dropless_mixture_experts_warp_gb300 import muon
    shapes = [(64, 96), (2, 300, 200), (129, 257)]
    for products in PRODUCTS:
        eager = run_step(shapes, steps=3, products=products)[0]
        p = run_step(shapes, steps=1, products=products)[0]
        p.workspace.fill_(0xff)                                          # NaN in every number
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            muon.step(p, lr=LR, momentum=MU, rms=RMS)
        graph.replay()
        p.workspace.fill_(0xff)
        graph.replay()
        muon.check(p)
        assert all(torch.equal(a, b) for a, b in zip(p.weights + p.m, eager.weights + eager.m))
