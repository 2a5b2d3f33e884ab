"""Refusals of the orthogonalised step that its ranges and its buffers ask for: on the host, before a launch (CPU)."""
import pytest
import torch
import torch

from test_blocks_refusals import B, P, muon_hyper, muon_table, status  # noqa: F401


def test_floor(B):  # noqa: F811
    run = lambda floor: status(B, "moe_muon_step_with", muon_hyper(B), muon_table(B), 1, floor, 1, P, 1 << 30, None, P)  # noqa: E731
    for floor in (-1e-9, float("nan"), float("inf"), 1e39):
        assert run(floor) == 1, floor
    assert status(B, "moe_muon_step_with", muon_hyper(B), muon_table(B, batch=-1), 1, 1e-7, 1, P, 1 << 30, None, P) == 1
    assert B.moe_muon_step_with(muon_hyper(B), muon_table(B), 0, 1e-7, 1, None, 0, None, P, stream=0) == 0


def test_products(B):  # noqa: F811
    """Operands in two parts need a workspace of their own size; other kinds are refused."""
    from dropless_mixture_experts_warp_gb300 import muon
    t = muon_table(B)
    need = [B.moe_muon_workspace_size_with(t, 1, 0, kind) for kind in (0, 1)]
    assert need[0] == B.moe_muon_workspace_size(t, 1, 0) < need[1]
    for kind in (0, 1):
        assert status(B, "moe_muon_step_with", muon_hyper(B), t, 1, 0.0, kind, P, need[kind] - 1, None, P) == 4
        assert B.moe_muon_workspace_size_with(t, 1, 1 << 30, kind) == 2 * need[kind]
    for kind in (-1, 2):
        assert status(B, "moe_muon_step_with", muon_hyper(B), t, 1, 0.0, kind, P, 1 << 30, None, P) == 1
        assert B.moe_muon_workspace_size_with(t, 1, 0, kind) == 0
    z = [torch.zeros(4, 5)]
    for make in (lambda: muon.plan(z, [torch.zeros(4, 5)], products="bf16"), lambda: muon.workspace([(4, 5)], device="cpu", products=1)):
        with pytest.raises(ValueError, match="products"):
            make()


def test_numbers_as_the_kernels_use_them(B):  # noqa: F811
    """A momentum that is 1 in fp32, decays and lengths of updates that are not finite there."""
    run = lambda h, t: status(B, "moe_muon_step", h, t, 1, P, 1 << 30, None, P)  # noqa: E731
    assert run(muon_hyper(B, momentum=1.0 - 1e-12), muon_table(B)) == 1
    assert run(muon_hyper(B, rms=3e38), muon_table(B)) == 1                  # times sqrt(16)
    for decay in (float("nan"), float("inf"), 1e39):
        assert run(muon_hyper(B), muon_table(B, weight_decay=decay)) == 1


def test_plans_of_tensors_that_share_memory(B):  # noqa: F811
    """Steps write weights, momenta and copies: none may share memory with anything, gradients only with each other."""
    from dropless_mixture_experts_warp_gb300 import muon
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)  # noqa: E731
    both = z(3, 4, 5)
    low = z(2, 4, 5, dt=torch.bfloat16)
    w, g, m = ([z(2, 4, 5) for _ in range(2)] for _ in range(3))
    for plan in (lambda: muon.plan(w, g, copies=[low, low]), lambda: muon.plan(w, g, copies=[low[:1].expand(2, 4, 5).contiguous(), None], m=[w[1], m[1]]),
                 lambda: muon.plan([both[:2], both[1:]], g), lambda: muon.plan(w, g, m=[both[:2], both[1:]]), lambda: muon.plan(w, [w[1], g[1]]),
                 lambda: muon.plan(w, g, m=[g[0], m[1]]), lambda: muon.plan([both[0]], [both[0]]),
                 lambda: muon.plan([z(4, 5)], [low[0]], copies=[low[0]])):
        with pytest.raises(ValueError, match="shares memory"):
            plan()
    muon.plan([both[:1], both[1:]], [g[0][:1], g[0]], copies=[None, low], m=[z(1, 4, 5), m[1]])     # neighbours; gradients share


def test_outputs_that_share_memory(B, monkeypatch):  # noqa: F811
    from dropless_mixture_experts_warp_gb300 import muon
    calls = []
    monkeypatch.setattr(muon.B, "check_device", lambda *a: None)
    monkeypatch.setattr(muon.B, "moe_muon_step_with", lambda *a: calls.append(a))
    both = torch.zeros(3, 4, 5)
    ws = muon.workspace([(2, 4, 5), (2, 4, 5)], device="cpu")
    x, o = ([torch.zeros(2, 4, 5) for _ in range(2)] for _ in range(2))
    low = torch.zeros(4, 4, 5, dtype=torch.bfloat16)
    for xs, outs in [(x, [o[0], o[0]]), (x, [both[:2], both[1:]]), (x, [x[1], o[1]]), ([both[:2], x[1]], [both[1:], o[1]]),
                     ([low[:2], x[1]], [low.view(-1).view(torch.float32).view(2, 4, 5), o[1]])]:
        with pytest.raises(ValueError, match="shares memory|contiguous"):
            muon.orthogonalize(xs, outs, ws)
    assert not calls
    for xs, outs in [(x, o), (x, x), ([x[0], x[0]], o), ([x[0], x[1]], [o[0], x[1]])]:
        muon.orthogonalize(xs, outs, ws)
    assert len(calls) == 4
