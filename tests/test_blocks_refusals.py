"""Refusals of the 8-bit products with blocks of 128 and of Muon: found on the host, before a launch (CPU); what their
early-launched kernels must keep to, from their sources."""
import ctypes
import os
import re

import pytest
import torch

P = 1 << 12     # an aligned address that nothing reads
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dropless_mixture_experts_warp_gb300", "csrc")


@pytest.fixture(scope="module")
def B():
    from dropless_mixture_experts_warp_gb300 import build, binding
    build.build()
    return binding


def status(B, fn, *args):
    before = B.moe_launch_count()
    with pytest.raises(B.MoeError) as e:
        getattr(B, fn)(*args, stream=0)
    assert B.moe_launch_count() == before
    return e.value.status


def changed(names, ok):
    return lambda **change: [change.get(n, v) for n, v in zip(names.split(), ok)]


def test_quantize(B):
    a = changed("src rows C row_map nrows codes scales codes_t scales_t", [P, 4, 128, None, None, P, P, P, P])
    for change, want in [(dict(rows=-1), 1), (dict(C=0), 1), (dict(src=None), 1), (dict(codes=None), 1), (dict(scales_t=None), 1),
                         (dict(codes=None, scales=None, codes_t=None, scales_t=None), 1), (dict(C=120), 2), (dict(rows=1 << 31), 2),
                         (dict(src=P + 2), 3), (dict(codes=P + 8), 3), (dict(codes_t=P + 8), 3)]:
        assert status(B, "moe_fp8_quantize", *a(**change)) == want, change
    assert B.moe_fp8_quantize(*a(rows=0), stream=0) == 0                   # nothing to do
    w = changed("src E N K codes codes_t scales", [P, 2, 128, 256, P, P, P])
    for change, want in [(dict(E=0), 1), (dict(N=-16), 1), (dict(src=None), 1), (dict(scales=None), 1), (dict(codes=None, codes_t=None), 1),
                         (dict(N=136), 2), (dict(K=8), 2), (dict(codes_t=P + 4), 3)]:
        assert status(B, "moe_fp8_quantize_weights", *w(**change)) == want, change


def test_products(B):
    a = changed("a sa rows K b sb turned N E offsets out status", [P, P, 4, 128, P, P, 0, 64, 2, P, P, P])
    for change, want in [(dict(rows=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(E=0), 1), (dict(offsets=None), 1), (dict(a=None), 1),
                         (dict(sa=None), 1), (dict(b=None), 1), (dict(sb=None), 1), (dict(out=None), 1), (dict(status=None), 1),
                         (dict(K=120), 2), (dict(N=68), 2), (dict(E=1025), 2), (dict(rows=1 << 31), 2), (dict(N=1 << 30, E=4), 2),
                         (dict(a=P + 8), 3), (dict(b=P + 1), 3), (dict(out=P + 2), 3)]:
        assert status(B, "moe_fp8_gemm", *a(**change)) == want, change
    assert B.moe_fp8_gemm(*a(rows=0), stream=0) == 0
    g = changed("dy sdy x sx rows N K E offsets out status", [P, P, P, P, 256, 16, 32, 2, P, P, P])
    for change, want in [(dict(rows=-128), 1), (dict(N=0), 1), (dict(offsets=None), 1), (dict(dy=None), 1), (dict(sx=None), 1), (dict(out=None), 1),
                         (dict(status=None), 1), (dict(rows=200), 2), (dict(K=20), 2), (dict(E=2000), 2), (dict(x=P + 4), 3), (dict(sx=P + 4), 3),
                         (dict(out=P + 2), 3)]:
        assert status(B, "moe_fp8_wgrad", *g(**change)) == want, change


def test_swiglu(B):
    a = changed("gu w rows f nrows codes scales", [P, P, 4, 64, None, P, P])
    for change, want in [(dict(rows=-1), 1), (dict(f=0), 1), (dict(gu=None), 1), (dict(scales=None), 1), (dict(f=24), 2), (dict(gu=P + 2), 3)]:
        assert status(B, "moe_fp8_swiglu", *a(**change)) == want, change
    g = changed("gu dh w rows f nrows c s ct st h hs dw part", [P, P, P, 4, 128, None, P, P, P, P, P, P, P, P])
    for change, want in [(dict(rows=-1), 1), (dict(dw=None), 1), (dict(part=None), 1), (dict(dh=None), 1), (dict(h=None), 1), (dict(f=64), 2),
                         (dict(ct=P + 8), 3)]:
        assert status(B, "moe_fp8_swiglu_bwd", *g(**change)) == want, change


def test_permute(B):
    dims = B.make_dims(4, 128, 128, 8, 2, prec="fp8-block")
    assert B.moe_check_dims(dims) == 0 and B.moe_check_dims(B.make_dims(4, 128, 64, 8, 2, prec="fp8-block")) == 2
    assert B.moe_check_dims(B.make_dims(4, 128, 128, 8, 2, prec=4)) == 1
    a = changed("x idx w split ro ws c s ct st r2t t2r wr status", [P] * 14)
    for change, want in [(dict(c=None), 1), (dict(st=None), 1), (dict(x=None), 1), (dict(status=None), 1), (dict(ws=None), 4), (dict(x=P + 2), 3)]:
        assert status(B, "moe_permute_fp8", dims, *a(**change)) == want, change


def muon_table(B, **change):
    t = (B.moe_muon_tensor * 1)()
    for n, v in {**dict(grad=P, m=P, w=P, w16=P, out=None, batch=2, rows=8, cols=16, weight_decay=0.0, grad_type=0, out_type=0), **change}.items():
        setattr(t[0], n, v)
    return t


def muon_hyper(B, **change):
    h = B.moe_muon_hyper(lr=1e-3, momentum=0.9, rms=0.2, nesterov=1, steps=1)
    h.coefficients[0:3] = [1.5, -0.5, 0.0]
    for n, v in change.items():
        setattr(h, n, v)
    return h


def test_muon(B):
    good = muon_table(B)
    need = B.moe_muon_workspace_size(good, 1, 0)
    assert need > 0 and B.moe_muon_workspace_size(good, 1, 1 << 30) == 2 * need
    run = lambda h, t, n=1, ws=P, size=1 << 30, st=P: status(B, "moe_muon_step", h, t, n, ws, size, None, st)  # noqa: E731
    for change in [dict(lr=-1.0), dict(lr=float("nan")), dict(lr=1e39), dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=float("nan")),
                   dict(rms=-1.0), dict(rms=float("inf")), dict(steps=0), dict(steps=17)]:
        assert run(muon_hyper(B, **change), good) == 1, change
    h = muon_hyper(B)
    h.coefficients[1] = float("inf")
    assert run(h, good) == 1
    h = muon_hyper(B)
    assert run(None, good) == 1 and run(h, good, st=None) == 1 and run(h, good, n=-1) == 1
    for change, want in [(dict(batch=-1), 1), (dict(rows=0), 1), (dict(cols=-3), 1), (dict(rows=1 << 17), 2), (dict(batch=1 << 25, rows=128), 2),
                         (dict(grad_type=2), 1), (dict(out_type=-1), 1), (dict(grad=None), 1), (dict(m=None), 1), (dict(w=None), 1),
                         (dict(out=P), 1), (dict(m=None, w=None), 1), (dict(m=None, w=None, out=P), 1)]:
        assert run(h, muon_table(B, **change)) == want, change              # the last: a bf16 copy without weights
    assert run(h, good, ws=None) == 4 and run(h, good, size=need - 1) == 4 and run(h, good, ws=P + 8) == 3
    assert B.moe_muon_step(h, good, 0, None, 0, None, P, stream=0) == 0     # nothing to do
    assert B.moe_muon_step(h, muon_table(B, batch=0), 1, None, 0, None, P, stream=0) == 0


def test_python_checks():
    """Shapes, types and devices, before the library is called: tensors on the CPU are refused."""
    from dropless_mixture_experts_warp_gb300 import fp8, layer, muon
    for bad in [(4, 100), (4, 0), (-1, 128)]:
        with pytest.raises(ValueError):
            fp8.allocate_rows(*bad, device="cpu")
    with pytest.raises(ValueError):
        fp8.allocate_weights(1, 24, 128, device="cpu")
    a, w = fp8.allocate_rows(5, 256, both=True, device="cpu"), fp8.allocate_weights(2, 128, 256, device="cpu")
    assert a.scales.shape == (2, 5) and a.codes_t.shape == (256, 128) and w.scales.shape == (2, 1, 2)
    with pytest.raises(ValueError):
        fp8.rows_of(a.codes)                                                # codes without scales
    with pytest.raises(ValueError):
        fp8.rows_of(a.codes, a.scales.t().contiguous())
    with pytest.raises(ValueError):
        fp8.weights_of(w.codes, w.scales[:, :, :1])
    with pytest.raises(ValueError):
        fp8.weights_of(w.codes, w.scales, codes_t=w.codes)
    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    for call in (lambda: fp8.quantize(a, x), lambda: fp8.quantize_weights(w, torch.zeros(2, 128, 256, dtype=torch.bfloat16)),
                 lambda: fp8.matmul(a, w, torch.zeros(5, 128, dtype=torch.bfloat16)),
                 lambda: fp8.weight_grad(a, a, torch.zeros(1, 256, 256, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            call()                                                          # not on a GPU
    g = [torch.zeros(3, 4, 5)]
    with pytest.raises(ValueError):
        muon.plan([torch.zeros(7)], [torch.zeros(7)])                       # not a matrix
    with pytest.raises(ValueError):
        muon.plan(g, [torch.zeros(3, 5, 4)])
    with pytest.raises(ValueError):
        muon.plan(g, [g[0].double()])
    with pytest.raises(ValueError):
        muon.plan(g, g, coefficients=[])
    with pytest.raises(ValueError):
        muon.plan(g, g, coefficients=[(1.0, 2.0)])
    with pytest.raises(ValueError):
        muon.plan(g, g, copies=[g[0]])
    with pytest.raises(ValueError):
        muon.plan(g, g, m=[None])
    with pytest.raises(ValueError):
        muon.plan(g * 2, [torch.zeros(3, 4, 5) for _ in range(2)])          # a weight twice
    b = layer.allocate(layer.dims_of(4, 128, 128, 4, 2, prec="fp8-block"), device="cpu", train=False)
    with pytest.raises(ValueError):
        layer.use_weights(b, w, w)
    with pytest.raises(ValueError):
        layer.use_weights(layer.allocate(layer.dims_of(4, 128, 128, 4, 2), device="cpu"), w, w)


def code(name):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)


@pytest.mark.parametrize("name", ["fp8_quant.cu", "fp8_gemm.cu", "muon.cu", "fp8.cuh", "pipe.cuh"])
def test_memory_may_change_while_an_early_kernel_waits(name):
    for word in ("__restrict__", "__ldg", ".nc."):
        assert word not in code(name), f"{name}: {word}"


@pytest.mark.parametrize("name", ["fp8_quant.cu", "fp8_gemm.cu", "muon.cu"])
def test_each_kernel_waits_once_and_before_it_lets_the_next_come_up(name):
    kernels = re.split(r"__global__", code(name))[1:]
    assert kernels
    for k in kernels:
        assert k.count("wait_for_previous()") == 1 and k.count("launch_dependents()") == 1, k[:100]
        assert k.index("wait_for_previous()") < k.index("launch_dependents()")


def test_structs_match_the_header():
    """ctypes' layouts of the two new structs against the C compiler's order and sizes."""
    from dropless_mixture_experts_warp_gb300 import binding as B
    assert ctypes.sizeof(B.moe_muon_tensor) == 5 * 8 + 6 * 4 and B.moe_muon_tensor.batch.offset == 40
    assert ctypes.sizeof(B.moe_muon_hyper) == 3 * 8 + 2 * 4 + 48 * 4 and B.moe_muon_hyper.coefficients.offset == 32
