"""The stack of blocks: its gradients against automatic differentiation in float64, and a short training (GPU)."""
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def reference(model, h, picks, target, score, offsets, k):
    """The stack in float64 on the CPU with the device's expert choices; gradients of the loss by autograd."""
    c = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
    norm = lambda x, w: x / (x.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    h0 = c(h)
    norms = [c(w) for w in model.norms]
    blocks = [{n: c(model.low[i][n] if n in model.low[i] else b[n]) for n in b} for i, b in enumerate(model.blocks)]
    stream, aux = h0, 0.0
    x = norm(stream, norms[0])
    for i, b in enumerate(blocks):
        logits = x @ b["router"].t()
        E = logits.shape[1]
        idx = picks[i]
        s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
        chosen = s.gather(1, idx)
        wts = chosen / chosen.sum(1, keepdim=True)
        y = torch.zeros_like(x)
        f = b["gu"].shape[1] // 2
        for e in range(E):
            t, j = (idx == e).nonzero(as_tuple=True)
            gu = x[t] @ b["gu"][e].t()
            act = torch.nn.functional.silu(gu[:, :f]) * gu[:, f:] * wts[t, j][:, None]
            y = y.index_add(0, t, act @ b["down"][e].t())
        p = s / s.sum(1, keepdim=True)
        for a, z in zip(offsets, offsets[1:]):
            load = torch.bincount(idx[a:z].reshape(-1), minlength=E).double() * E / (k * (z - a))
            aux = aux + model.coef * (load * p[a:z].mean(0)).sum() / (len(offsets) - 1)
        aux = aux + model.z_coef * torch.logsumexp(logits, 1).square().mean()
        stream = stream + b["gate"] * norm(y, b["post"])
        x = norm(stream, norms[i + 1])
    loss = (x - target.double().cpu()).square().mean() + aux
    leaves = [h0] + [b[n] for b in blocks for n in ("gu", "down", "router", "post", "gate")] + norms
    return x.detach(), torch.autograd.grad(loss, leaves)


@pytest.mark.parametrize("score,stream", [("softmax", "bf16"), ("sigmoid", "fp32")])
def test_gradients(score, stream):
    """Relative error of whole tensors.  A bf16 rounding is at most 2^-8 and the path from the loss back to the first
    block's weights has at most 16 of them (two blocks: the stream, x, G|U, h, y, dy, dG|dU, dx each): 16 * 2^-8 = 6 %
    were they all to agree in sign."""
    from dropless_mixture_experts_warp_gb300 import train
    T, d, f, E, k = 384, 128, 64, 8, 2
    offsets = [0, 100, 101, 384]
    # large aux coefficients: their gradients have to show beside the loss's
    model = train.Stack(T, d, f, E, k, score=score, stream=stream, sequences=3, coef=1.0, z_coef=0.1)
    h = torch.randn(T, d, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(model.stream)
    target = torch.randn(T, d, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    x = model.forward(h, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    dh = model.backward((2 * (x.float() - target) / (T * d)).bfloat16())
    model.check()
    got = [dh]
    for i in range(2):
        got += [model.bufs[i].dw_gu, model.bufs[i].dw_d, model.d_router[i], model.merges[i].dw_post, model.merges[i].dgate]
    got += [model.pre.dw, model.merges[0].dw, model.merges[1].dw]
    picks = [b.topk_idx.long().cpu() for b in model.bufs]
    want_x, want = reference(model, h, picks, target, score, offsets, k)
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(x, want_x) < 0.03
    for a, b in zip(got, want):
        assert rel(a, b) < 0.06


@pytest.mark.parametrize("bits", [32, 8])
def test_training_lowers_the_loss(bits):
    from dropless_mixture_experts_warp_gb300 import train
    T, d, f, E, k = 512, 256, 128, 8, 2
    model = train.Stack(T, d, f, E, k, bits=bits)
    g = torch.Generator("cuda").manual_seed(5)
    h = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    target = torch.tanh(h.float() @ (torch.randn(d, d, device="cuda", generator=g) / 16))
    losses = []
    for t in range(1, 41):
        off = model.forward(h).float() - target
        losses.append(float(off.square().mean()))
        model.backward((2 * off / off.numel()).bfloat16())
        model.update(t, lr=3e-3)
    model.check()
    assert losses[-1] < 0.5 * losses[0]
