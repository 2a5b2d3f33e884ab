"""Refusals of the operators around the layer: found on the host, before anything is launched (CPU)."""
import pytest


@pytest.fixture(scope="module")
def B():
    from dropless_mixture_experts_warp_gb300 import build, binding
    build.build()
    return binding


P = 1 << 12     # an aligned address that nothing reads


def status(B, fn, *args):
    before = B.moe_launch_count()
    with pytest.raises(B.MoeError) as e:
        getattr(B, fn)(*args, stream=0)
    assert B.moe_launch_count() == before
    return e.value.status


def test_norm_dims(B):
    good = dict(T=4, d=64)
    assert B.moe_norm_check_dims(B.make_norm_dims(**good)) == 0
    for bad, want in [(dict(T=-1), 1), (dict(d=0), 1), (dict(d=68), 2), (dict(d=16392), 2), (dict(eps=0.0), 1),
                      (dict(eps=float("nan")), 1)]:
        dims = B.make_norm_dims(**{**good, **bad})
        assert B.moe_norm_check_dims(dims) == want, bad
        assert B.moe_norm_workspace_size(dims) == 0
        assert status(B, "moe_norm_fwd", dims, P, P, P) == want
    for field, value in [("stream_type", 2), ("weight_type", -1), ("gate", 3), ("gate_act", 2)]:
        dims = B.make_norm_dims(**good)
        setattr(dims, field, value)
        assert B.moe_norm_check_dims(dims) == 1, field


def test_norm_and_merge_arguments(B):
    dims = B.make_norm_dims(4, 64)
    assert status(B, "moe_norm_fwd", dims, None, P, P) == 1
    assert status(B, "moe_norm_fwd", dims, P + 8, P, P) == 3
    assert status(B, "moe_norm_bwd", dims, P, P, P, None, P, None, P) == 1
    assert status(B, "moe_norm_bwd", dims, P, P, P, None, P, P, None) == 4
    assert status(B, "moe_norm_bwd", dims, P, P, P, P + 2, P, P, P) == 3
    # h, y, w_post, gate, w_next, h_out, x_next
    assert status(B, "moe_merge_fwd", dims, P, P, P, P, P, P, P) == 1          # a gate without a gate kind
    assert status(B, "moe_merge_fwd", dims, P, P, P, None, None, P, P) == 1    # x_next without w_next
    assert status(B, "moe_merge_fwd", dims, P, P, P, None, P, P, None) == 1    # w_next without x_next
    assert status(B, "moe_merge_fwd", dims, P, P, P, None, P, P, P + 4) == 3
    # dh_out, dx_next, h_out, y, w_post, gate, w_next, dh, dy, dw_post, dgate, dw_next, workspace
    ok = [P, P, P, P, P, None, P, P, P, P, None, P, P]

    def bwd(dims, **change):
        names = ["dh_out", "dx_next", "h_out", "y", "w_post", "gate", "w_next", "dh", "dy", "dw_post", "dgate", "dw_next",
                 "workspace"]
        return status(B, "moe_merge_bwd", dims, *[change.get(n, v) for n, v in zip(names, ok)])

    assert bwd(dims, dw_post=None) == 1
    assert bwd(dims, w_next=None) == 1
    assert bwd(dims, dx_next=None) == 1
    assert bwd(dims, h_out=None) == 1
    assert bwd(dims, dgate=P) == 1
    assert bwd(dims, y=None) == 1
    assert bwd(dims, workspace=None) == 4
    assert bwd(dims, dy=P + 8) == 3
    assert bwd(dims, w_next=None, dw_next=None, dx_next=None, dh_out=None) == 1   # no gradient at all
    for gate in ("channel", "token"):
        assert bwd(B.make_norm_dims(4, 64, gate=gate), gate=P) == 1            # no dgate


def test_balance_dims_and_arguments(B):
    good = dict(T=64, E=8, k=2)
    assert B.moe_balance_check_dims(B.make_balance_dims(**good)) == 0
    for bad, want in [(dict(T=-1), 1), (dict(E=0), 1), (dict(k=9), 1), (dict(k=0), 1), (dict(E=64, k=33), 1),
                      (dict(sequences=0), 1), (dict(E=1025), 2), (dict(sequences=65536), 2),
                      (dict(coef=float("inf")), 1), (dict(z_coef=float("nan")), 1)]:
        dims = B.make_balance_dims(**{**good, **bad})
        assert B.moe_balance_check_dims(dims) == want, bad
        assert B.moe_balance_workspace_size(dims) == 0
    one, two = B.make_balance_dims(**good), B.make_balance_dims(sequences=2, **good)
    # logits, topk_idx, seq_offsets, mask, losses, counts, prob_mean, seq_tokens, workspace, dev_status
    assert status(B, "moe_balance_fwd", one, None, P, None, None, P, P, P, P, P, P) == 1
    assert status(B, "moe_balance_fwd", one, P, P, None, None, None, P, P, P, P, P) == 1
    assert status(B, "moe_balance_fwd", one, P, P, None, None, P, P, P, P, P, None) == 1
    assert status(B, "moe_balance_fwd", one, P, P, None, None, P, P, P, P, None, P) == 4
    assert status(B, "moe_balance_fwd", one, P + 4, P, None, None, P, P, P, P, P, P) == 3
    assert status(B, "moe_balance_fwd", two, P, P, None, None, P, P, P, P, P, P) == 1
    # logits, seq_offsets, mask, counts, seq_tokens, grad_losses, accumulate, d_logits
    assert status(B, "moe_balance_bwd", one, P, None, None, None, P, None, 1, P) == 1
    assert status(B, "moe_balance_bwd", one, P, None, None, P, P, None, 1, None) == 1
    assert status(B, "moe_balance_bwd", two, P, None, None, P, P, None, 1, P) == 1
    assert status(B, "moe_balance_bwd", one, P, None, None, P, P, None, 1, P + 8) == 3


def test_adamw_arguments(B):
    import ctypes

    def step(change=None, hyper=None, count=2, bits=32):
        h = B.moe_adamw_hyper(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=0, bits=bits)
        for k, v in (hyper or {}).items():
            setattr(h, k, v)
        t = (B.moe_adamw_tensor * 2)()
        for i in range(2):
            t[i] = B.moe_adamw_tensor(P, P, P, P, P, P if bits == 8 else None, P if bits == 8 else None, 100, 0.1, 0)
        for k, v in (change or {}).items():
            setattr(t[1], k, v)
        return status(B, "moe_adamw_step", h, t, count, None)

    for field, value, want in [("w", None, 1), ("grad", None, 1), ("m", None, 1), ("v", None, 1), ("n", -1, 1),
                               ("grad_type", 2, 1), ("m_scale", P, 1), ("weight_decay", float("inf"), 1),
                               ("w", P + 4, 3), ("w16", P + 2, 3), ("grad", P + 8, 3), ("m", P + 1, 3)]:
        assert step({field: value}) == want, field
    for field, value, want in [("m_scale", None, 1), ("v_scale", None, 1), ("v_scale", P + 2, 3), ("v", P + 4, 3)]:
        assert step({field: value}, bits=8) == want, field
    for field, value in [("lr", -1.0), ("lr", float("nan")), ("beta1", 1.0), ("beta2", -0.1), ("eps", 0.0), ("step", 0),
                         ("bits", 16)]:
        assert step(hyper={field: value}) == 1, field
    assert step(count=-1) == 1
    h = B.moe_adamw_hyper(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=0, bits=32)
    assert status(B, "moe_adamw_step", h, None, 1, None) == 1
    assert status(B, "moe_adamw_step", None, None, 0, None) == 1
    t = (B.moe_adamw_tensor * 1)(B.moe_adamw_tensor(None, None, None, P, P, P, P, 100, 0.0, 0))
    out = lambda p: (ctypes.c_void_p * 1)(p)  # noqa: E731
    assert status(B, "moe_adamw_values", t, 1, 2, out(P), out(P)) == 1
    assert status(B, "moe_adamw_values", t, 1, 0, out(None), out(P)) == 1
    assert status(B, "moe_adamw_values", t, 1, 0, out(P), out(P + 4)) == 3
    t[0].m_scale = None
    assert status(B, "moe_adamw_values", t, 1, 0, out(P), out(P)) == 1


def test_adamw_plan_refuses_tensors_that_do_not_fit(B):
    import torch
    from dropless_mixture_experts_warp_gb300 import optim
    w = torch.zeros(8, 16)
    good = dict(weights=[w], grads=[w.clone()])
    p = optim.plan(**good, bits=8)
    assert p.m[0].dtype == torch.int8 and p.v_scale[0].shape == (1,)
    for bad in (dict(grads=[w.half()]), dict(grads=[w[:4]]), dict(grads=[w.t()]), dict(grads=[]), dict(copies=[w]),
                dict(bits=16), dict(weights=[w.bfloat16()]), dict(m=[w.double()]), dict(weight_decay=[0.0, 0.0]),
                dict(m_scale=[torch.zeros(1)]), dict(bits=8, m_scale=[torch.zeros(2)])):
        with pytest.raises(ValueError):
            optim.plan(**{**good, **bad})
    with pytest.raises(ValueError):
        optim.values(optim.plan(**good))


def test_adamw_refuses_tensors_that_are_not_on_one_gpu(B):
    import torch
    from dropless_mixture_experts_warp_gb300 import optim
    w = torch.zeros(8, 16)
    p = optim.plan([w], [w.clone()], bits=8)
    for call in (lambda: optim.step(p, lr=1e-3, step=1), lambda: optim.values(p)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="device"):
        optim.plan([w, w.to("meta")], [w, w.to("meta")])
    with pytest.raises(ValueError):
        optim.plan([w], [None])
    with pytest.raises(ValueError):
        optim.plan([w], [w], m=[None])


def test_lists_of_tensors_are_checked_one_by_one(B):
    import torch
    ts = [torch.zeros(3, 4), torch.zeros(5)]
    shapes, cpu = [t.shape for t in ts], torch.device("cpu")
    B.check_tensors(ts, torch.float32, shapes, cpu)
    B.check_tensors([], torch.float32, [], cpu)
    for bad in ([ts[0]], [ts[0], None], [ts[1], ts[0]], [ts[0].t().contiguous().t(), ts[1]], [ts[0], ts[1].double()],
                [ts[0], ts[1].to("meta")]):
        with pytest.raises(ValueError):
            B.check_tensors(bad, torch.float32, shapes, cpu)


def test_adamw_eps_and_lr_are_checked_as_the_kernels_have_them(B):
    """In fp32: an eps that rounds to 0 there would make 0 / 0 of an element without a gradient, and with 8-bit states
    one below the root of the smallest v that they hold would divide by next to nothing; lr must not become infinite."""

    def step(bits, **hyper):
        h = B.moe_adamw_hyper(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=0, bits=bits), **hyper})
        s = P if bits == 8 else None
        t = (B.moe_adamw_tensor * 1)(B.moe_adamw_tensor(P, P, P, P, P, s, s, 100, 0.1, 0))
        return status(B, "moe_adamw_step", h, t, 1, None)

    for bits in (32, 8):
        for eps in (1e-50, 2.0 ** -151, 1e39, float("inf"), float("nan"), -1e-8):
            assert step(bits, eps=eps) == 1, (bits, eps)
        for lr in (1e39, float("inf")):
            assert step(bits, lr=lr) == 1, (bits, lr)
    for eps in (1e-40, 1e-38, 1e-20, 2.0 ** -63 * (1 - 2.0 ** -20)):
        assert step(8, eps=eps) == 1, eps
    # what is still taken: no tensors, so that nothing is launched
    before = B.moe_launch_count()
    for bits, eps in ((32, 1e-40), (32, 1e-45), (8, 2.0 ** -63), (8, 1e-15)):
        h = B.moe_adamw_hyper(lr=1e-3, beta1=0.9, beta2=0.99, eps=eps, step=1, seed=0, bits=bits)
        B.moe_adamw_step(h, None, 0, None, stream=0)
    assert B.moe_launch_count() == before


def test_buffers_on_another_device_are_refused(B, monkeypatch):
    """Buffers on the CPU, or on a GPU that is not the current one (here told by a stand-in for its query)."""
    import dataclasses
    import types

    import torch
    from dropless_mixture_experts_warp_gb300 import balance, block, optim
    bf = torch.bfloat16
    n = block.allocate(block.dims_of(4, 64), device="cpu")
    h, w = torch.zeros(4, 64, dtype=bf), torch.ones(64)
    o = balance.allocate(4, 8, 2, device="cpu")
    l, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    far = types.SimpleNamespace(device=torch.device("cuda:1"))      # of a tensor its device alone is looked at
    p = optim.plan([torch.zeros(8)], [torch.zeros(8)], bits=8)

    def calls(n, o, p, **kw):
        return (lambda: block.norm_forward(n, h, w, **kw), lambda: block.norm_backward(n, h, h, w, **kw),
                lambda: block.merge_forward(n, h, h, w_next=w, **kw), lambda: block.merge_backward(n, h, h, h, h, w_next=w, **kw),
                lambda: balance.forward(o, l, idx, **kw), lambda: balance.backward(o, l, l.clone(), **kw),
                lambda: optim.step(p, lr=1e-3, step=1, **kw), lambda: optim.values(p, **kw))

    before = B.moe_launch_count()
    for call in calls(n, o, p, stream=0):
        with pytest.raises(ValueError, match="runs on a GPU"):
            call()
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    away = dataclasses.replace(p, device=torch.device("cuda:1"))
    for call in calls(dataclasses.replace(n, x=far), dataclasses.replace(o, losses=far), away, stream=0):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            call()
    B.check_device(torch.device("cuda:0"), 0)
    here = types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=0)
    B.check_device(torch.device("cuda:0"), here)
    with pytest.raises(ValueError, match="stream"):
        B.check_device(torch.device("cuda:0"), types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0))
    # a step's control elsewhere than its tensors
    near = dataclasses.replace(p, device=torch.device("cuda:0"))
    with pytest.raises(ValueError, match="expected a contiguous"):
        optim.step(near, lr=1e-3, step=1, control=optim.Control(device="cpu"), stream=0)
    assert B.moe_launch_count() == before


def test_the_balance_gradient_gets_the_forwards_coefficients(B, monkeypatch):
    """The dims that reach the entry points, without a GPU: both calls replaced."""
    import torch
    from dropless_mixture_experts_warp_gb300 import balance
    seen = []
    note = lambda dims, *a: seen.append((dims.coef, dims.z_coef))  # noqa: E731
    monkeypatch.setattr(B, "moe_balance_fwd", note)
    monkeypatch.setattr(B, "moe_balance_bwd", note)
    monkeypatch.setattr(B, "check_device", lambda *a: None)
    o = balance.allocate(4, 8, 2, device="cpu")
    l, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    balance.backward(o, l, l.clone())
    balance.forward(o, l, idx, coef=0.5, z_coef=0.25)
    balance.backward(o, l, l.clone())
    balance.backward(o, l, l.clone(), coef=2.0)
    balance.backward(o, l, l.clone(), z_coef=0.0)
    balance.backward(o, l, l.clone())
    balance.forward(o, l, idx)
    balance.backward(o, l, l.clone())
    assert seen == [(1.0, 0.0), (0.5, 0.25), (0.5, 0.25), (2.0, 0.25), (0.5, 0.0), (0.5, 0.25), (1.0, 0.0), (1.0, 0.0)]
