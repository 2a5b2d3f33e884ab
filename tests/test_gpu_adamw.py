"""AdamW steps over lists of tensors against the float64 form, 32-bit and 8-bit states (GPU)."""
import numpy as np
import pytest
import torch

from oracle import around as oa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

U = oa.U32
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def tensors(sizes, seed=0, scale=1e-2):
    rng = np.random.default_rng(seed)
    out = []
    for n in sizes:
        w, g = rng.standard_normal(n), rng.standard_normal(n) * scale
        m, v = rng.standard_normal(n) * scale, (rng.standard_normal(n) * scale) ** 2
        out.append(dict(w=w, g=g, m=m, v=v))
    return out


def cuda(x, kind=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(kind).cuda()


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, majorant, terms, half=0.0):
    """Within `terms` roundings of 2^-24 on the majorant and one of `half` on the value."""
    assert np.all(abs(got - ref) <= half * abs(ref) + (1 + half) * terms * U * majorant + 1e-37)


def check_step(before, w, m, v, wd, t, got_w, got_m, got_v, gs=1.0, lr_scale=1.0):
    """Four roundings make m, five v; the update's root, quotients and bias corrections (each within 2 units, the
    corrections of 1 - beta^t from the device's step within 8) and v's error under the root: 32 on the update."""
    h = {**HYPER, "lr": HYPER["lr"] * lr_scale}
    w1, m1, v1 = oa.adamw(w, before["g64"], m, v, t=t, wd=wd, grad_scale=gs, **h)
    g = gs * before["g64"]
    mm = HYPER["beta1"] * abs(m) + (1 - HYPER["beta1"]) * abs(g)
    vm = HYPER["beta2"] * v + (1 - HYPER["beta2"]) * g * g
    if got_m is not None:
        close(got_m, m1, mm, 8)
        close(got_v, v1, vm, 8)
    update = mm / (1 - HYPER["beta1"] ** t) / (np.sqrt(v1 / (1 - HYPER["beta2"] ** t)) + HYPER["eps"])
    close(got_w, w1, abs(w) + h["lr"] * (update + wd * abs(w)), 32)
    return m1, v1, mm, vm


@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [127, 128, 129, 4095, 4096, 4097], [5000, 1, 70001, 12],
                                   list(range(1, 250))])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_32_bit(sizes, grad):
    from dropless_mixture_experts_warp_gb300 import optim
    ts = tensors(sizes)
    ws, gs = [cuda(t["w"]) for t in ts], [cuda(t["g"], grad) for t in ts]
    copies = [None if i % 3 == 1 else torch.zeros_like(w, dtype=torch.bfloat16) for i, w in enumerate(ws)]
    decay = [0.1 * (i % 2) for i in range(len(ts))]
    ms, vs = [cuda(t["m"]) for t in ts], [cuda(t["v"]) for t in ts]
    p = optim.plan(ws, gs, copies=copies, weight_decay=decay, m=ms, v=vs)
    old = [[f64(x) for x in (w, m, v)] for w, m, v in zip(ws, ms, vs)]
    optim.step(p, step=7, **HYPER)
    for i, t in enumerate(ts):
        t["g64"] = f64(gs[i])
        check_step(t, *old[i], decay[i], 7, f64(ws[i]), f64(ms[i]), f64(vs[i]))
        if copies[i] is not None:
            assert torch.equal(copies[i], ws[i].bfloat16())


@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [127, 128, 129, 4095, 4096, 4097], [5000, 1, 70001, 12],
                                   list(range(1, 250))])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_8_bit(sizes, grad):
    """Codes equal the definition's, except where a draw lies within fp32's roundings of the border between two."""
    from dropless_mixture_experts_warp_gb300 import optim
    ts = tensors(sizes, 1)
    ws, gs = [cuda(t["w"]) for t in ts], [cuda(t["g"], grad) for t in ts]
    copies = [torch.zeros_like(w, dtype=torch.bfloat16) for w in ws]
    rng = np.random.default_rng(2)
    ms = [cuda(rng.integers(-127, 128, n), torch.int8) for n in sizes]
    vs = [cuda(rng.integers(0, 256, n), torch.uint8) for n in sizes]
    sm = [cuda(1e-2 * (0.5 + rng.random(-(-n // 128)))) for n in sizes]
    sv = [cuda(1e-4 * (0.5 + rng.random(-(-n // 128)))) for n in sizes]
    p = optim.plan(ws, gs, copies=copies, bits=8, weight_decay=0.1, m=ms, v=vs, m_scale=sm, v_scale=sv)
    old = [(f64(ws[i]), oa.decode(f64(ms[i]), f64(sm[i]), 127, 2), oa.decode(f64(vs[i]), f64(sv[i]), 255, 4))
           for i in range(len(sizes))]
    optim.step(p, step=5, seed=123, **HYPER)
    mv, vv = optim.values(p, dtype=torch.float32)
    mb, vb = optim.values(p)
    for i, t in enumerate(ts):
        t["g64"] = f64(gs[i])
        m1, v1, mm, vm = check_step(t, *old[i], 0.1, 5, f64(ws[i]), None, None)
        assert torch.equal(copies[i], ws[i].bfloat16())
        for x, maj, s, code, draw, top, power, val, low in ((m1, mm, sm, ms, 0, 127, 2, mv, mb), (v1, vm, sv, vs, 1, 255, 4, vv, vb)):
            scales = f64(s[i])
            ref = oa.block_scales(x)
            # 16 roundings: the decoded state's 5, the moment's 5 and their products
            limit = 16 * U * oa.block_scales(maj)
            assert np.all(abs(scales - ref) <= limit)
            draws = oa.adamw_draws(123, 5, i, sizes[i])[draw]
            want, margin = oa.encode(x, ref, draws, top, power)
            got = code[i].cpu().numpy().astype(np.int64)
            # the share's roundings (24 of them) over the width of a code there, times the block's largest majorant
            k = np.maximum(abs(want) - 1, 0)
            width = ((k + 1) / top) ** power - (k / top) ** power
            rep = np.repeat(np.divide(oa.block_scales(maj), ref, out=np.ones_like(ref), where=ref > 0), 128)[:sizes[i]]
            near = margin <= 24 * U * rep / width
            assert np.array_equal(got[~near], want[~near])
            assert np.all(abs(got - want) <= 1)
            close(f64(val[i]), oa.decode(got, scales, top, power), abs(oa.decode(got, scales, top, power)), 8)
            assert torch.equal(low[i], val[i].bfloat16())


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_from_zero_train(bits):
    """100 steps on a quadratic: both kinds of state bring the loss down to the same order, step for step repeatable."""
    from dropless_mixture_experts_warp_gb300 import optim
    target = torch.linspace(-1, 1, 1000, device="cuda")
    runs = []
    for _ in range(2):
        w, g = torch.zeros(1000, device="cuda"), torch.zeros(1000, device="cuda")
        p = optim.plan([w], [g], bits=bits)
        for t in range(1, 101):
            torch.sub(w, target, out=g)
            optim.step(p, lr=2e-2, step=t, seed=11)
        runs.append(w.clone())
    assert torch.equal(runs[0], runs[1])
    assert float((runs[0] - target).square().mean()) < 0.05 * float(target.square().mean())


@pytest.mark.parametrize("bits", [32, 8])
def test_control_and_capture(bits):
    """A captured step replayed with new values in device memory is the step with those values; skip changes nothing."""
    from dropless_mixture_experts_warp_gb300 import optim
    sizes = [300, 4097]
    ts = tensors(sizes, 3)

    def fresh():
        ws, gs = [cuda(t["w"]) for t in ts], [cuda(t["g"]) for t in ts]
        return optim.plan(ws, gs, copies=[torch.zeros_like(w, dtype=torch.bfloat16) for w in ws], bits=bits)

    state = lambda p: p.weights + p.copies + p.m + p.v + ((p.m_scale + p.v_scale) if bits == 8 else [])  # noqa: E731
    p, c = fresh(), optim.Control()
    start = [x.clone() for x in state(p)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        optim.step(p, step=0, seed=5, control=c, **HYPER)
    for x, y in zip(state(p), start):
        assert torch.equal(x, y)               # capturing runs nothing
    c.skip.fill_(1)
    p.grads[0].fill_(float("nan"))
    g.replay()
    for x, y in zip(state(p), start):
        assert torch.equal(x, y)
    p.grads[0].copy_(cuda(ts[0]["g"]))
    c.skip.fill_(0)
    old = [[f64(w), np.zeros(n), np.zeros(n)] for w, n in zip(p.weights, sizes)]
    for t, gs, ls in ((1, 0.5, 1.0), (2, 2.0, 0.25)):
        c.step.fill_(t)
        c.grad_scale.fill_(gs)
        c.lr_scale.fill_(ls)
        g.replay()
        if bits == 8:
            ms, vs = optim.values(p, dtype=torch.float32)
        else:
            ms, vs = p.m, p.v
        for i, x in enumerate(ts):
            x["g64"] = f64(p.grads[i])
            exact = bits == 32
            check_step(x, *old[i], 0.0, t, f64(p.weights[i]), f64(ms[i]) if exact else None, f64(vs[i]) if exact else None,
                       gs=gs, lr_scale=ls)
            old[i] = [f64(p.weights[i]), f64(ms[i]), f64(vs[i])]


def test_blocks_of_zeros_and_of_numbers_fp32_cannot_scale():
    from dropless_mixture_experts_warp_gb300 import optim
    w = torch.ones(384, device="cuda")
    g = torch.zeros(384, device="cuda")
    g[128:256] = 1e-38                          # m below the smallest normal number, v below any
    g[256:] = 1e-15                             # v = 5e-32 (a normal number)
    p = optim.plan([w], [g], bits=8)
    for t in (1, 2):
        optim.step(p, step=t, **HYPER)
    assert torch.isfinite(w).all() and torch.equal(w[:128], torch.ones(128, device="cuda"))
    assert torch.count_nonzero(p.m[0][:256]) == 0 and p.m_scale[0][:2].tolist() == [0.0, 0.0]
    assert torch.all(p.v[0][256:] == 255) and torch.all(p.m[0][256:] == 127)


def test_side_stream():
    from dropless_mixture_experts_warp_gb300 import optim
    ts = tensors([9000], 4)
    out = []
    for stream in (None, torch.cuda.Stream()):
        w, g = cuda(ts[0]["w"]), cuda(ts[0]["g"])
        p = optim.plan([w], [g], bits=8)
        torch.cuda.synchronize()
        optim.step(p, step=1, stream=stream, **HYPER)
        torch.cuda.synchronize()
        out.append((w, p.m[0], p.v[0], p.m_scale[0], p.v_scale[0]))
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("bits", [32, 8])
def test_large_tensors(bits):
    """Units of several blocks a warp: sampled elements (whole blocks of 128) of 21M against the definition."""
    from dropless_mixture_experts_warp_gb300 import optim
    n = 21_000_001
    g = torch.Generator("cuda").manual_seed(8)
    r = lambda: torch.randn(n, device="cuda", generator=g)  # noqa: E731
    w, grad = r(), r().mul_(1e-2).bfloat16()
    small = torch.randn(77, device="cuda", generator=g)
    ws, gs = [w, small], [grad, torch.full((77,), 1e-2, device="cuda")]
    if bits == 32:
        p = optim.plan(ws, gs, weight_decay=0.1, m=[r().mul_(1e-2), torch.zeros(77, device="cuda")],
                       v=[r().mul_(1e-2).square_(), torch.zeros(77, device="cuda")])
    else:
        blocks = -(-n // 128)
        p = optim.plan(ws, gs, weight_decay=0.1, bits=8)
        p.m[0].copy_(torch.randint(-127, 128, (n,), device="cuda", generator=g))
        p.v[0].copy_(torch.randint(0, 256, (n,), device="cuda", generator=g))
        p.m_scale[0].copy_(torch.rand(blocks, device="cuda", generator=g) * 1e-2 + 1e-3)
        p.v_scale[0].copy_(torch.rand(blocks, device="cuda", generator=g) * 1e-4 + 1e-6)
    pick = np.unique(np.concatenate([np.arange(64), np.random.default_rng(1).integers(0, n // 128, 3000), [n // 128]]))
    at = np.minimum((pick[:, None] * 128 + np.arange(128)), n - 1)
    inside = (pick[:, None] * 128 + np.arange(128)) < n
    take = lambda t: f64(t[torch.from_numpy(at.ravel()).cuda()]).reshape(at.shape) * inside  # noqa: E731
    rows = lambda t: f64(t[torch.from_numpy(pick).cuda()])  # noqa: E731
    old_w, g64 = take(w), take(grad)
    if bits == 32:
        old_m, old_v = take(p.m[0]), take(p.v[0])
    else:
        k, q = take(p.m[0]), take(p.v[0])
        old_m = rows(p.m_scale[0])[:, None] * np.sign(k) * (k / 127) ** 2
        old_v = rows(p.v_scale[0])[:, None] * (q / 255) ** 4
    optim.step(p, step=3, seed=77, **HYPER)
    exact = bits == 32
    m1, v1, mm, vm = check_step({"g64": g64}, old_w, old_m, old_v, 0.1, 3, take(w), take(p.m[0]) if exact else None,
                                take(p.v[0]) if exact else None)
    if exact:
        return
    draws = [oa.adamw_draws(77, 3, 0, n)[i][at.ravel()].reshape(at.shape) for i in (0, 1)]
    for x, maj, code, scale, u, top, power in ((m1, mm, p.m[0], p.m_scale[0], draws[0], 127, 2),
                                               (v1, vm, p.v[0], p.v_scale[0], draws[1], 255, 4)):
        s = (abs(x) * inside).max(axis=1)
        big = maj.max(axis=1)
        assert np.all(abs(rows(scale) - s) <= 16 * U * big)
        want, margin = oa.encode((x * inside).ravel(), s, u.ravel(), top, power)
        want, margin = want.reshape(at.shape), margin.reshape(at.shape)
        got = take(code)
        low = np.maximum(abs(want) - 1, 0)
        width = ((low + 1) / top) ** power - (low / top) ** power
        near = margin <= 24 * U * (big / s)[:, None] / width
        assert np.array_equal(got[~near], want[~near])
        assert np.all(abs(got - want) <= 1)


@pytest.mark.parametrize("scale", [1e-17, 1e-10, 1e15])
def test_8_bit_at_far_scales(scale):
    """Codes follow the definition where the inverse of a scale, or a share's product, would leave fp32's range."""
    from dropless_mixture_experts_warp_gb300 import optim
    n = 4096
    rng = np.random.default_rng(12)
    w, g = torch.zeros(n, device="cuda"), cuda(rng.standard_normal(n) * scale * 10.0 ** rng.uniform(-3, 0, n))
    p = optim.plan([w], [g], bits=8)
    optim.step(p, step=1, seed=4, **HYPER)
    g64 = f64(g)
    m1, v1 = (1 - HYPER["beta1"]) * g64, (1 - HYPER["beta2"]) * g64 ** 2
    for x, code, scales, u, top, power in ((m1, p.m[0], p.m_scale[0], 0, 127, 2), (v1, p.v[0], p.v_scale[0], 1, 255, 4)):
        ref = oa.block_scales(x)
        assert np.all(abs(f64(scales) - ref) <= 8 * U * ref)
        want, margin = oa.encode(x, ref, oa.adamw_draws(4, 1, 0, n)[u], top, power)
        got = code.cpu().numpy().astype(np.int64)
        low = np.maximum(abs(want) - 1, 0)
        # the roundings are relative to the value; a v below fp32's normal numbers is rounded to 2^-149, or to 0
        largest = np.repeat(ref, 128)
        width = ((low + 1) / top) ** power - (low / top) ** power
        near = (margin <= (24 * U * abs(x) + 2.0 ** -149) / largest / width) | ((x != 0) & (abs(x) < 2.0 ** -149))
        assert np.array_equal(got[~near], want[~near]) and np.all(abs(got - want) <= 1)
        assert near.mean() < 0.2


@pytest.mark.parametrize("wd", [0.1, 0.02])
@pytest.mark.parametrize("bits", [32, 8])
def test_small_decay_is_not_lost_in_rounding(bits, wd):
    """lr * wd of 1e-7 and 2e-8, near and below the distance of 1 from its neighbours: the drift of the mean weight
    against the same steps without decay.  Weights lie in [1, 2), so a step rounds each by at most 2^-24, as good as
    uniformly (the updates spread over several units): two runs of K steps leave the mean of n differences a deviation
    of 2^-23 / sqrt(12) * sqrt(2 K / n), of which 6 are allowed.  The weights themselves move by less than K lr."""
    from dropless_mixture_experts_warp_gb300 import optim
    n, lr, warm, K = 1 << 18, 1e-6, 5, 50
    start = 1 + torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    ends = []
    for decay in (wd, 0.0):
        rng = torch.Generator("cuda").manual_seed(6)
        w, g = start.clone(), torch.zeros(n, device="cuda")
        p = optim.plan([w], [g], bits=bits, weight_decay=decay)
        for t in range(1, warm + K + 1):       # the first steps only fill the moments (step 1 moves by lr exactly)
            g.normal_(generator=rng).mul_(1e-3)
            optim.step(p, lr=lr if t > warm else 0.0, step=t, beta1=0.5, beta2=0.95, seed=9)
        ends.append(w.double())
    drift = float((ends[0] - ends[1]).mean())
    want = -K * lr * wd * float(start.double().mean())
    assert abs(drift - want) <= 6 * 2.0 ** -23 / 12 ** 0.5 * (2 * K / n) ** 0.5 + abs(want) * 2 * K * lr


def test_8_bit_at_scales_near_the_largest_number():
    """Codes follow the definition where the inverse of a block's scale is below fp32's normal numbers."""
    from dropless_mixture_experts_warp_gb300 import optim
    n = 1000
    rng = np.random.default_rng(13)
    w, g = torch.zeros(n, device="cuda"), cuda(rng.standard_normal(n) * 1e10)
    ms, vs = cuda(rng.integers(-127, 128, n), torch.int8), cuda(rng.integers(1, 256, n), torch.uint8)
    sm, sv = (cuda(3e38 * (0.5 + 0.5 * rng.random(-(-n // 128)))) for _ in range(2))
    p = optim.plan([w], [g], bits=8, m=[ms], v=[vs], m_scale=[sm], v_scale=[sv])
    old_m, old_v = oa.decode(f64(ms), f64(sm), 127, 2), oa.decode(f64(vs), f64(sv), 255, 4)
    optim.step(p, step=3, seed=4, **HYPER)
    m1, v1, mm, vm = check_step({"g64": f64(g)}, np.zeros(n), old_m, old_v, 0.0, 3, f64(w), None, None)
    for x, maj, code, scales, u, top, power in ((m1, mm, ms, sm, 0, 127, 2), (v1, vm, vs, sv, 1, 255, 4)):
        ref = oa.block_scales(x)
        assert ref.min() > 2.0 ** 126                # the case is what it says
        assert np.all(abs(f64(scales) - ref) <= 16 * U * oa.block_scales(maj))
        want, margin = oa.encode(x, ref, oa.adamw_draws(4, 3, 0, n)[u], top, power)
        got = code.cpu().numpy().astype(np.int64)
        k = np.maximum(abs(want) - 1, 0)
        width = ((k + 1) / top) ** power - (k / top) ** power
        near = margin <= 24 * U * np.repeat(oa.block_scales(maj) / ref, 128)[:n] / width
        assert np.array_equal(got[~near], want[~near]) and np.all(abs(got - want) <= 1)
        assert near.mean() < 0.2


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_written_just_before_and_on_another_stream(bits, captured):
    """The step comes up while what precedes it runs: gradients and control values that a slow kernel or another
    stream's copies write count all the same, and what follows may overwrite them."""
    from dropless_mixture_experts_warp_gb300 import optim
    n, wd = 300_001, 0.1
    t = tensors([n], 9)[0]
    first, second = cuda(t["g"]), cuda(t["m"])

    def fresh():
        w, g = cuda(t["w"]), torch.full((n,), 3.0, device="cuda")
        return optim.plan([w], [g], copies=[torch.zeros_like(w, dtype=torch.bfloat16)], bits=bits, weight_decay=wd), optim.Control()

    state = lambda p: p.weights + p.copies + p.m + p.v + ((p.m_scale + p.v_scale) if bits == 8 else [])  # noqa: E731
    p, c = fresh()
    for step, g in ((1, first), (2, second)):
        p.grads[0].copy_(g)
        c.step.fill_(step)
        torch.cuda.synchronize()
        optim.step(p, step=0, seed=5, control=c, **HYPER)
        torch.cuda.synchronize()
    want = [x.clone() for x in state(p)]
    if bits == 8:
        want += [x.clone() for x in sum(optim.values(p), [])]
    p, c = fresh()
    start = [x.clone() for x in state(p)]
    got = [torch.zeros_like(x) for x in want]
    values = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()

    def fill(step, g):
        torch.cuda._sleep(200_000)
        p.grads[0].copy_(g)
        c.step.fill_(step)

    def work():
        here = torch.cuda.current_stream()
        for x, y in zip(state(p), start):
            x.copy_(y)
        fill(1, first)
        optim.step(p, step=0, seed=5, control=c, **HYPER)
        p.grads[0].fill_(3.0)
        c.step.fill_(9)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            fill(2, second)
        here.wait_stream(side)
        optim.step(p, step=0, seed=5, control=c, **HYPER)
        if bits == 8:
            optim.values(p, values[:1], values[1:])
        p.grads[0].fill_(3.0)
        for x, y in zip(got, state(p) + values):
            x.copy_(y)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    s.synchronize()
    if captured:
        for x in got:
            x.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            work()
        torch.cuda.synchronize()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
