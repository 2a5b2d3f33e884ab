"""Block norms and merges against the float64 forms, forward and backward (GPU)."""
import numpy as np
import pytest
import torch

from oracle import around as oa
from tests.around_util import DTYPE, check, dev
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

# Roundings between an input and a row's result: a thread adds up to 32 elements, then two trees of 5 sums; the
# root, the products and (sigmoid) the exponential, whose error is at most 2 + |x| units, take fewer than 64 more.
ROW = 128


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def inputs(T, d, stream, weights, seed=0):
    rng = np.random.default_rng([T, d, seed])
    r = rng.standard_normal
    out = {"h": dev(r((T, d)) * 2, stream), "y": dev(r((T, d)) * 0.4, "bf16"), "w": dev(1 + 0.2 * r(d), weights),
           "w_post": dev(0.5 + 0.2 * r(d), weights), "dh": dev(r((T, d)), stream), "dx": dev(r((T, d)), "bf16"),
           "channel": dev(r(d), weights), "token": dev(r(T), "fp32"), "none": (None, None)}
    return out


SHAPES = [(1, 8), (2, 16), (5, 504), (33, 512), (4, 520), (700, 128), (1, 7168), (311, 2056), (7, 8192), (6, 8200),
          (3, 16384)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("stream,weights", [("bf16", "fp32"), ("fp32", "bf16")])
def test_norm(T, d, stream, weights):
    from dropless_mixture_experts_warp_gb300 import block
    b = block.allocate(block.dims_of(T, d, stream=stream, weights=weights, eps=1e-6, weight_offset=1.0))
    i = inputs(T, d, stream, weights)
    (h, h64), (w, w64), (dx, dx64), (add, add64) = i["h"], i["w"], i["dx"], i["dh"]
    x = oa.norm_fwd(h64, w64, 1e-6, 1.0)
    check("x", block.norm_forward(b, h, w), (x, abs(x)), "bf16", ROW)
    ref = oa.norm_bwd(dx64, h64, w64, 1e-6, 1.0, add64)
    block.norm_backward(b, dx, h, w, dh_add=add)
    check("dh", b.dh, ref["dh"], stream, ROW)
    check("dw", b.dw, ref["dw"], "fp32", T + ROW)
    ref = oa.norm_bwd(dx64, h64, w64, 1e-6, 1.0)
    first = block.norm_backward(b, dx, h, w).clone(), b.dw.clone()
    check("dh alone", b.dh, ref["dh"], stream, ROW)
    block.norm_backward(b, dx, h, w)
    assert torch.equal(first[0], b.dh) and torch.equal(first[1], b.dw), "two calls differ"


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("stream,weights", [("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("gate,act,post,nxt", [("none", "identity", True, True), ("channel", "identity", True, True),
                                               ("channel", "sigmoid", False, True), ("token", "sigmoid", True, False),
                                               ("token", "identity", False, True), ("none", "identity", False, False)])
def test_merge(T, d, stream, weights, gate, act, post, nxt):
    from dropless_mixture_experts_warp_gb300 import block
    scales = dict(alpha=0.75, beta=1.25)
    dims = block.dims_of(T, d, stream=stream, weights=weights, gate=gate, gate_act=act, eps=1e-5, **scales)
    b = block.allocate(dims)
    i = inputs(T, d, stream, weights, 1)
    opt = dict(eps=1e-5, kind=gate, sigmoid=act == "sigmoid", alpha=0.75, beta=1.25)
    w_post, w_next = i["w_post"] if post else (None, None), i["w"] if nxt else (None, None)
    ref = oa.merge_fwd(i["h"][1], i["y"][1], w_post[1], i[gate][1], w_next[1], **opt)
    block.merge_forward(b, i["h"][0], i["y"][0], w_post=w_post[0], gate=i[gate][0], w_next=w_next[0])
    check("h_out", b.h_out, ref["h_out"], stream, ROW)
    if nxt:
        check("x", b.x, ref["x"], "bf16", 2 * ROW)
    # the stream that the backward sees is any stream: h itself
    ref = oa.merge_bwd(i["dh"][1], i["dx"][1], i["h"][1], i["y"][1], w_post[1], i[gate][1], w_next[1], **opt)
    args = (i["dh"][0], i["dx"][0] if nxt else None, i["h"][0], i["y"][0])
    kw = dict(w_post=w_post[0], gate=i[gate][0], w_next=w_next[0])
    block.merge_backward(b, *args, **kw)
    got = {"dh": b.dh, "dy": b.dy, "dw_post": b.dw_post, "dgate": b.dgate, "dw_next": b.dw}
    kind = {"dh": stream, "dy": "bf16"}
    terms = {"dh": ROW, "dy": 3 * ROW, "dw_next": T + ROW, "dw_post": T + 2 * ROW,
             "dgate": (d if gate == "token" else T) + 3 * ROW}
    for name in ref:
        check(name, got[name], ref[name], kind.get(name, "fp32"), terms[name])
    kept = {n: got[n].clone() for n in ref}
    block.merge_backward(b, *args, **kw)
    assert all(torch.equal(kept[n], got[n]) for n in ref), "two calls differ"


def test_gradient_of_the_next_norm_alone():
    """dh_out None: the gradient reaches the stream through the next norm only."""
    from dropless_mixture_experts_warp_gb300 import block
    b = block.allocate(block.dims_of(9, 264, eps=1e-6))
    i = inputs(9, 264, "bf16", "fp32")
    ref = oa.merge_bwd(None, i["dx"][1], i["h"][1], i["y"][1], None, None, i["w"][1], eps=1e-6)
    block.merge_backward(b, None, i["dx"][0], i["h"][0], None, w_next=i["w"][0])
    check("dh", b.dh, ref["dh"], "bf16", ROW)
    check("dy", b.dy, ref["dy"], "bf16", ROW)


@pytest.mark.parametrize("d", [512, 520])
def test_no_tokens(d):
    from dropless_mixture_experts_warp_gb300 import block
    b = block.allocate(block.dims_of(0, d, gate="channel"))
    i = inputs(0, d, "bf16", "fp32")
    for t in (b.dw, b.dw_post, b.dgate):
        t.fill_(7.0)
    block.norm_forward(b, i["h"][0], i["w"][0])
    block.merge_forward(b, i["h"][0], i["y"][0], w_post=i["w_post"][0], gate=i["channel"][0], w_next=i["w"][0])
    block.merge_backward(b, i["dh"][0], i["dx"][0], i["h"][0], i["y"][0], w_post=i["w_post"][0], gate=i["channel"][0],
                         w_next=i["w"][0])
    for t in (b.dw, b.dw_post, b.dgate):
        assert torch.count_nonzero(t) == 0


@pytest.mark.parametrize("d", [256, 4096])
def test_rows_of_zeros_and_of_infinities_keep_to_themselves(d):
    from dropless_mixture_experts_warp_gb300 import block
    T = 40
    i = inputs(T, d, "fp32", "fp32")
    h, y = i["h"][0], i["y"][0]
    h[3] = 0
    y[3] = 0
    clean = block.allocate(block.dims_of(T, d, stream="fp32"))
    block.merge_forward(clean, h, y, w_post=i["w_post"][0], w_next=i["w"][0])
    assert torch.count_nonzero(clean.x[3]) == 0 and torch.isfinite(clean.x).all()
    h2, y2 = h.clone(), y.clone()
    h2[5, 1], y2[6, d - 1] = float("nan"), float("inf")
    b = block.allocate(clean.dims)
    block.merge_forward(b, h2, y2, w_post=i["w_post"][0], w_next=i["w"][0])
    others = [t for t in range(T) if t not in (5, 6)]
    assert torch.equal(b.x[others], clean.x[others]) and torch.equal(b.h_out[others], clean.h_out[others])
    assert not torch.isfinite(b.x[5]).any() and not torch.isfinite(b.h_out[6, d - 1])


@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_in_place_and_on_another_stream(stream):
    from dropless_mixture_experts_warp_gb300 import binding as B, block
    T, d = 129, 1040
    i = inputs(T, d, stream, "fp32")
    dims = block.dims_of(T, d, stream=stream, gate="token", gate_act="sigmoid")
    b = block.allocate(dims)
    w = dict(w_post=i["w_post"][0], gate=i["token"][0], w_next=i["w"][0])
    block.merge_forward(b, i["h"][0], i["y"][0], **w)
    block.merge_backward(b, i["dh"][0], i["dx"][0], b.h_out, i["y"][0], **w)
    other = block.allocate(dims)
    side = torch.cuda.Stream()
    h, dh = i["h"][0].clone(), i["dh"][0].clone()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_merge_fwd(dims, h, i["y"][0], *w.values(), h, other.x, side)
    B.moe_merge_bwd(dims, dh, i["dx"][0], h, i["y"][0], *w.values(), dh, other.dy, other.dw_post, other.dgate,
                    other.dw, other.workspace, side)
    side.synchronize()
    assert torch.equal(h, b.h_out) and torch.equal(other.x, b.x) and torch.equal(dh, b.dh)
    for n in ("dy", "dw_post", "dgate", "dw"):
        assert torch.equal(getattr(other, n), getattr(b, n)), n


def test_captured_steps_replay():
    from dropless_mixture_experts_warp_gb300 import block
    T, d = 65, 2048
    i = inputs(T, d, "bf16", "fp32")
    b = block.allocate(block.dims_of(T, d))
    w = dict(w_post=i["w_post"][0], w_next=i["w"][0])
    block.merge_forward(b, i["h"][0], i["y"][0], **w)
    block.merge_backward(b, i["dh"][0], i["dx"][0], b.h_out, i["y"][0], **w)
    want = [t.clone() for t in (b.h_out, b.x, b.dh, b.dy, b.dw, b.dw_post)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block.merge_forward(b, i["h"][0], i["y"][0], **w)
        block.merge_backward(b, i["dh"][0], i["dx"][0], b.h_out, i["y"][0], **w)
    for t in (b.h_out, b.x, b.dh, b.dy, b.dw, b.dw_post):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, t) for a, t in zip(want, (b.h_out, b.x, b.dh, b.dy, b.dw, b.dw_post)))


def test_tensors_that_do_not_fit_are_refused():
    from dropless_mixture_experts_warp_gb300 import block
    b = block.allocate(block.dims_of(16, 64))
    h, w = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    for bad in (h.float(), h[:8], h.t().contiguous().t(), torch.zeros(16, 128, dtype=h.dtype, device="cuda")[:, ::2],
                h.cpu()):
        with pytest.raises(ValueError):
            block.norm_forward(b, bad, w)
    with pytest.raises(ValueError):
        block.norm_forward(b, h, w.bfloat16())
    with pytest.raises(ValueError):
        block.merge_forward(b, h, h, gate=w[:32], w_next=w)


# More rows than are under way at once, so that every group takes several: each kernel variant by its width
# (a warp, part of a block, a block a row; weights in shared memory or not; units that end inside the row)
LONG = [(5300, 512), (5000, 264), (1300, 1040), (1100, 4096), (950, 7168), (620, 8200), (330, 16384)]


@pytest.mark.parametrize("T,d", LONG)
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_many_rows(T, d, stream):
    from dropless_mixture_experts_warp_gb300 import block
    i = inputs(T, d, stream, "fp32", 2)
    (h, h64), (y, y64), (w, w64), (wp, wp64), (dx, dx64), (dh, dh64) = (i[n] for n in ("h", "y", "w", "w_post", "dx", "dh"))
    b = block.allocate(block.dims_of(T, d, stream=stream))
    x = oa.norm_fwd(h64, w64, 1e-6)
    check("x", block.norm_forward(b, h, w), (x, abs(x)), "bf16", ROW)
    ref = oa.norm_bwd(dx64, h64, w64, 1e-6, 0.0, dh64)
    block.norm_backward(b, dx, h, w, dh_add=dh)
    check("dh", b.dh, ref["dh"], stream, ROW)
    check("dw", b.dw, ref["dw"], "fp32", T + ROW)
    for gate, act in (("none", "identity"), ("channel", "identity"), ("channel", "sigmoid"), ("token", "sigmoid")):
        b = block.allocate(block.dims_of(T, d, stream=stream, gate=gate, gate_act=act))
        opt = dict(eps=1e-6, kind=gate, sigmoid=act == "sigmoid")
        g, g64 = i[gate]
        ref = oa.merge_fwd(h64, y64, wp64, g64, w64, **opt)
        block.merge_forward(b, h, y, w_post=wp, gate=g, w_next=w)
        check("h_out", b.h_out, ref["h_out"], stream, ROW)
        check("x", b.x, ref["x"], "bf16", 2 * ROW)
        ref = oa.merge_bwd(dh64, dx64, h64, y64, wp64, g64, w64, **opt)
        block.merge_backward(b, dh, dx, h, y, w_post=wp, gate=g, w_next=w)
        got = {"dh": b.dh, "dy": b.dy, "dw_post": b.dw_post, "dgate": b.dgate, "dw_next": b.dw}
        terms = {"dh": ROW, "dy": 3 * ROW, "dw_next": T + ROW, "dw_post": T + 2 * ROW,
                 "dgate": (d if gate == "token" else T) + 3 * ROW}
        for n in ref:
            check(f"{gate} {act} {n}", got[n], ref[n], {"dh": stream, "dy": "bf16"}.get(n, "fp32"), terms[n])


# Widths at which the gradients' ring leaves the weights room only with one row of y fewer: units that fill the
# threads and that do not, and a width at which it does for one of the types alone
@pytest.mark.parametrize("T,d", [(800, 8192), (700, 7176), (900, 6664)])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_many_rows_of_wide_streams(T, d, stream):
    test_many_rows(T, d, stream)


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_written_just_before_and_on_another_stream(captured):
    """The kernels come up while what precedes them runs: they read nothing before it is done, be it a slow kernel
    of their stream, of another that it waits for, or a copy; and what follows may overwrite their inputs."""
    from dropless_mixture_experts_warp_gb300 import block
    T, d = 2048, 1024
    i = inputs(T, d, "bf16", "fp32", 3)
    (h, _), (w, _), (dx, _) = i["h"], i["w"], i["dx"]
    b = block.allocate(block.dims_of(T, d))
    want = block.norm_forward(b, h, w).clone()
    want_dh, want_dw = block.norm_backward(b, dx, h, w).clone(), b.dw.clone()
    src, dst, x, dh, dw = (torch.zeros_like(t) for t in (h, dx, want, want_dh, want_dw))
    side = torch.cuda.Stream()

    def work():
        here = torch.cuda.current_stream()
        torch.cuda._sleep(200_000)
        torch.mul(h, 1.0, out=src)
        x.copy_(block.norm_forward(b, src, w))
        src.zero_()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000)
            src.copy_(h)
            dst.copy_(dx)
        here.wait_stream(side)
        dh.copy_(block.norm_backward(b, dst, src, w))
        dw.copy_(b.dw)
        dst.zero_()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    s.synchronize()
    if captured:
        for t in (src, dst, x, dh, dw):
            t.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            work()
        torch.cuda.synchronize()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
    assert torch.equal(x, want) and torch.equal(dh, want_dh) and torch.equal(dw, want_dw)


@pytest.mark.parametrize("T,d", [(33, 512), (7, 7168), (40, 520), (6, 8200)])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("post", [True, False])
def test_gradients_of_gates_far_open_and_far_shut(T, d, stream, gate, post):
    """The sigmoid's slope where the gate is as good as 1 or 0: e^-|g|, which 1 - sigmoid(g) does not hold in fp32."""
    from dropless_mixture_experts_warp_gb300 import block
    b = block.allocate(block.dims_of(T, d, stream=stream, gate=gate, gate_act="sigmoid"))
    i = inputs(T, d, stream, "fp32", 4)
    far = np.random.default_rng(T + d).choice([-30.0, -16.0, -0.5, 15.0, 16.0, 17.5, 30.0], d if gate == "channel" else T)
    g, g64 = dev(far, "fp32")
    w_post = i["w_post"] if post else (None, None)
    opt = dict(eps=1e-6, kind=gate, sigmoid=True)
    ref = oa.merge_fwd(i["h"][1], i["y"][1], w_post[1], g64, i["w"][1], **opt)
    block.merge_forward(b, i["h"][0], i["y"][0], w_post=w_post[0], gate=g, w_next=i["w"][0])
    check("h_out", b.h_out, ref["h_out"], stream, ROW)
    ref = oa.merge_bwd(i["dh"][1], i["dx"][1], i["h"][1], i["y"][1], w_post[1], g64, i["w"][1], **opt)
    block.merge_backward(b, i["dh"][0], i["dx"][0], i["h"][0], i["y"][0], w_post=w_post[0], gate=g, w_next=i["w"][0])
    check("dy", b.dy, ref["dy"], "bf16", 3 * ROW)
    check("dgate", b.dgate, ref["dgate"], "fp32", (d if gate == "token" else T) + 3 * ROW)
