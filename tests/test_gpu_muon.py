"""The orthogonalised step on the GPU, against float64.

The products run on fp16 operands.  What that costs depends on the matrix, so the bound is its own: the same steps with
the same roundings in float64 (newton_schulz_rounded) are e off the exact ones, and the kernels, which round other
values in other places of those roundings (their fp32 sums differ in the last bits), may be 1.5 e off, and a rounding
of the result: half a step of its type (bf16 2^-8) of each value.
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def matrices(rng, b, m, n, kind, scale=1e-4):
    r = max(1, min(m, n) // 16)
    x = rng.standard_normal((b, m, r)) @ rng.standard_normal((b, r, n)) * (2.0 / np.sqrt(r)) + rng.standard_normal((b, m, n))
    return torch.from_numpy(x * scale).to(kind)


def near(got, x, kind):
    """got within the bound of the orthogonal factor of x (float64 [m, n])."""
    ref = ob.newton_schulz(x)
    low = ob.newton_schulz_rounded(x)
    e = np.linalg.norm((low.T if x.shape[0] > x.shape[1] else low) - ref)
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.linalg.norm(got - ref)
    assert off <= 1.5 * e + (HALF[kind] + 2.0 ** -20) * np.linalg.norm(ref), (off / max(np.linalg.norm(ref), 1e-30), e)


SHAPES = [(1, 1, 1), (2, 16, 40), (3, 131, 72), (1, 128, 128), (2, 129, 257), (1, 300, 700), (2, 512, 1024), (1, 640, 384),
          (5, 7, 200), (1, 1, 300)]


@pytest.mark.parametrize("b,m,n", SHAPES)
@pytest.mark.parametrize("kind,out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
def test_orthogonalize(b, m, n, kind, out):
    from dropless_mixture_experts_warp_gb300 import muon
    x = matrices(np.random.default_rng(m + n), b, m, n, kind)
    w = muon.workspace([x.shape])
    o = torch.full(x.shape, 7.0, dtype=out, device="cuda")
    muon.orthogonalize([x.cuda()], [o], w)
    muon.check(w)
    for i in range(b):
        near(o[i], x[i].double().numpy(), out)
    again = torch.empty_like(o)
    muon.orthogonalize([x.cuda()], [again], w)
    assert torch.equal(o, again)


def test_scale_zero_and_nan():
    """The result does not depend on the matrix's scale; a zero matrix gives zeros, a NaN stays in its matrix."""
    from dropless_mixture_experts_warp_gb300 import muon
    x = matrices(np.random.default_rng(1), 4, 96, 160, torch.float32, scale=1.0)
    x[1] = 0.0
    x[2, 5, 7] = float("nan")
    x[3] = x[0] * 2.0 ** -40
    w = muon.workspace([x.shape])
    o = torch.empty(x.shape, device="cuda")
    muon.orthogonalize([x.cuda()], [o], w)
    near(o[0], x[0].double().numpy(), torch.float32)
    assert (o[1] == 0).all() and torch.isnan(o[2]).all() and torch.equal(o[0], o[3])


def run_step(shapes, kind=torch.bfloat16, copies=True, nesterov=True, workspace=1 << 30, steps=2, control=None, seed=0):
    from dropless_mixture_experts_warp_gb300 import muon
    rng = np.random.default_rng(seed)
    ws, gs, ms = [], [], []
    for s in shapes:
        b = int(np.prod(s[:-2]))
        ws.append(torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.02).cuda())
        gs.append(matrices(rng, b, s[-2], s[-1], kind).reshape(s).cuda())
        ms.append(matrices(rng, b, s[-2], s[-1], torch.float32, 5e-4).reshape(s).cuda())
    low = [w.bfloat16() if copies else None for w in ws]
    start = [w.clone() for w in ws], [m.clone() for m in ms]
    p = muon.plan(ws, gs, copies=low, m=ms, weight_decay=[0.1 * (i + 1) for i in range(len(ws))], workspace=workspace)
    for _ in range(steps):
        muon.step(p, lr=2e-3, momentum=0.95, rms=0.2, nesterov=nesterov, control=control)
    muon.check(p)
    return p, start, gs, low


@pytest.mark.parametrize("kind,nesterov,copies", [(torch.bfloat16, True, True), (torch.float32, False, False)])
def test_step(kind, nesterov, copies):
    shapes = [(48, 80), (3, 131, 72), (2, 2, 48, 80), (131, 72), (256, 256)]
    p, (w0, m0), gs, low = run_step(shapes, kind, copies, nesterov, steps=1)
    lr, mu, rms = 2e-3, 0.95, 0.2
    for i, s in enumerate(shapes):
        m, n = s[-2:]
        flat = lambda t: t.double().cpu().numpy().reshape(-1, m, n)  # noqa: E731
        for w, mm, g, nw, nm in zip(flat(w0[i]), flat(m0[i]), flat(gs[i]), flat(p.weights[i]), flat(p.m[i])):
            ref, mref, o = ob.muon_step(w, mm, g, lr, mu, 0.1 * (i + 1), rms, nesterov)
            assert np.all(np.abs(nm - mref) <= 3 * ob.U32 * (np.abs(mu * mm) + np.abs(g)))      # fp32 momentum, one fma
            u = g + mu * mref if nesterov else mref
            e = np.linalg.norm((lambda r: r.T if m > n else r)(ob.newton_schulz_rounded(u)) - o)
            size = lr * rms * np.sqrt(max(m, n))
            off = np.linalg.norm(nw - ref)
            assert off <= size * (1.5 * e + 2.0 ** -11 * np.linalg.norm(o)) + 4 * ob.U32 * np.linalg.norm(np.abs(w) + size * np.abs(o))
        if copies:
            assert torch.equal(low[i], p.weights[i].bfloat16())


def test_chunks_and_many_tensors():
    """A workspace of one matrix and one of all give the same bits; more tensors of a shape than a launch takes."""
    shapes = [(40, 56)] * 70 + [(7, 40, 56), (130, 20), (3, 130, 20)]
    big = run_step(shapes)[0]
    small = run_step(shapes, workspace=1)[0]
    middle = run_step(shapes, workspace=700_000)[0]
    assert small.workspace.numel() < middle.workspace.numel() < big.workspace.numel()
    for other in (small, middle):
        for a, b, c, d in zip(big.weights, other.weights, big.m, other.m):
            assert torch.equal(a, b) and torch.equal(c, d)


def test_control():
    """Scales and skip are read on the device."""
    from dropless_mixture_experts_warp_gb300 import optim
    shapes = [(64, 96), (2, 33, 40)]
    c = optim.Control()
    c.skip.fill_(1)
    p, (w0, m0), _, _ = run_step(shapes, control=c)
    assert all(torch.equal(a, b) for a, b in zip(p.weights + p.m, w0 + m0))
    c.skip.fill_(0)
    same = run_step(shapes, control=c)[0]
    plain = run_step(shapes)[0]
    assert all(torch.equal(a, b) for a, b in zip(same.weights + same.m, plain.weights + plain.m))
    c.lr_scale.fill_(0.0)
    p, (w0, m0), _, _ = run_step(shapes, control=c)
    assert all(torch.equal(a, b) for a, b in zip(p.weights, w0)) and not any(torch.equal(a, b) for a, b in zip(p.m, m0))


def test_captured_step():
    """A captured step, replayed, gives the bits of eager ones."""
    from dropless_mixture_experts_warp_gb300 import muon
    shapes = [(64, 96), (2, 300, 200)]
    eager = run_step(shapes, steps=3)[0]
    p = run_step(shapes, steps=1)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        muon.step(p, lr=2e-3, momentum=0.95, rms=0.2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(p.weights + p.m, eager.weights + eager.m))
