"""Balance loss, counts, z-loss and their gradient against the float64 forms (GPU)."""
import numpy as np
import pytest
import torch

from oracle import around as oa
from tests.around_util import check
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

# Roundings of a row's result: 32 terms a lane and a tree of 5 sums, twice, and the exponentials, the logarithm and
# the quotients (at most 2 units each) around them.
ROW = 128
COEF, Z = 0.5, 0.25


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def case(T, E, k, S, masked, seed=0, spread=1.0):
    rng = np.random.default_rng([T, E, k, S, seed])
    l = (rng.standard_normal((T, E)) * spread + rng.standard_normal(E)).astype(np.float32)
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    cuts = np.sort(rng.integers(0, T + 1, S - 1))
    if S > 3:
        cuts[1] = cuts[0]                  # an empty sequence
    offsets = np.concatenate([[0], cuts, [T]]).astype(np.int32)
    mask = None
    if masked:
        mask = (rng.random(T) < 0.7).astype(np.uint8) * 3   # any value but 0 keeps a token
        if S > 1:
            mask[offsets[-2]:] = 0         # a sequence of padding alone
    return l, idx, offsets, mask


def cuda(*arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def run(l, idx, offsets, mask, score, k, z=Z):
    """Forward and backward on the device against the float64 forms."""
    from dropless_mixture_experts_warp_gb300 import balance
    T, E = l.shape
    S = len(offsets) - 1
    b = balance.allocate(T, E, k, score=score, sequences=S)
    dl, di, do, dm = cuda(l, idx, offsets, mask)
    if S == 1:
        do = None
    balance.forward(b, dl, di, seq_offsets=do, mask=dm, coef=COEF, z_coef=z)
    ref = oa.balance_fwd(l.astype(np.float64), idx, offsets, mask, k, score, COEF, z)
    assert np.array_equal(b.counts.cpu().numpy(), ref["counts"])
    assert np.array_equal(b.seq_tokens.cpu().numpy(), ref["seq_tokens"])
    # every term is positive, so the majorant is the value; an exponential near fp32's lowest normal numbers may be
    # flushed: 1e-37 of a row's sum, which `check` allows
    check("prob_mean", b.prob_mean, (ref["prob_mean"],) * 2, "fp32", T + ROW)
    check("losses", b.losses, (ref["losses"],) * 2, "fp32", T + S + E + 2 * ROW)
    balance.check(b)
    grad = np.array([1.5, -0.75], np.float32)
    d, m = oa.balance_bwd(l.astype(np.float64), offsets, mask, ref["counts"], ref["seq_tokens"], k, score, COEF, z, grad)
    out = torch.full((T, E), 7.0, device="cuda")
    balance.backward(b, dl, out, seq_offsets=do, mask=dm, coef=COEF, z_coef=z, grad=cuda(grad)[0], accumulate=False)
    check("d_logits", out, (d, m), "fp32", 2 * ROW)
    base = np.random.default_rng(5).standard_normal((T, E)).astype(np.float32) * 1e-3
    acc = cuda(base)[0]
    balance.backward(b, dl, acc, seq_offsets=do, mask=dm, coef=COEF, z_coef=z, grad=cuda(grad)[0])
    check("d_logits added", acc, (d + base, m + abs(base)), "fp32", 2 * ROW)
    if mask is not None:
        kept = torch.from_numpy(mask == 0).cuda()
        assert torch.equal(acc[kept], cuda(base)[0][kept]) and torch.count_nonzero(out[kept]) == 0
    first = [t.clone() for t in (b.losses, b.prob_mean, b.counts)]
    balance.forward(b, dl, di, seq_offsets=do, mask=dm, coef=COEF, z_coef=z)
    assert all(torch.equal(x, y) for x, y in zip(first, (b.losses, b.prob_mean, b.counts))), "two calls differ"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S,masked", [(1, 1, 1, 1, False), (1, 8, 2, 1, False), (7, 3, 3, 1, True), (257, 8, 2, 1, False),
                                            (1000, 60, 4, 5, True), (129, 64, 6, 40, True), (640, 65, 8, 3, False),
                                            (4111, 128, 8, 9, True), (3001, 256, 8, 2, False), (515, 300, 32, 4, True),
                                            (300, 1001, 8, 2, True), (200, 1024, 8, 1, False), (5, 512, 1, 7, False)])
def test_balance(T, E, k, S, masked, score):
    run(*case(T, E, k, S, masked), score, k)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_no_z_loss(score):
    run(*case(300, 32, 4, 3, True), score, 4, z=0.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_out_of_reach_and_rows_without_mass(score):
    l, idx, offsets, mask = case(400, 48, 4, 3, False, spread=8.0)
    l[:, 5] = -np.inf
    l[:, 7] = np.finfo(np.float32).min
    l[17] = -np.inf                        # nothing in reach
    l[18, :] = np.finfo(np.float32).min    # the type's lowest value everywhere: equal shares
    l[20] -= 150.0                         # sigmoids below fp32's range: the shares remain
    l[19, 3] = 300.0
    idx = np.argsort(-l, axis=1, kind="stable")[:, :4].astype(np.int32)
    # logsumexp of the lowest value squares to infinity, in fp32 and not in float64: without the z-loss
    run(l, idx, offsets, mask, score, 4, z=0.0)
    l[18] = -80.0
    run(l, idx, offsets, mask, score, 4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_tokens_may_hold_anything(score):
    from dropless_mixture_experts_warp_gb300 import balance
    l, idx, offsets, mask = case(700, 72, 4, 6, True)
    outs = []
    for fill in (0.0, np.nan, np.inf, -np.inf):
        x = l.copy()
        x[mask == 0] = fill
        j = idx.copy()
        j[mask == 0] = 10 ** 6             # not looked at
        b = balance.allocate(700, 72, 4, score=score, sequences=6)
        dl, di, do, dm = cuda(x, j, offsets, mask)
        balance.forward(b, dl, di, seq_offsets=do, mask=dm, coef=COEF, z_coef=Z)
        balance.check(b)
        d = torch.zeros(700, 72, device="cuda")
        balance.backward(b, dl, d, seq_offsets=do, mask=dm, coef=COEF, z_coef=Z)
        outs.append((b.losses, b.counts, b.prob_mean, d))
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, outs[0]))


def test_nothing_kept_and_no_tokens():
    from dropless_mixture_experts_warp_gb300 import balance
    for T, S in ((0, 1), (0, 3), (50, 3)):
        b = balance.allocate(T, 16, 2, sequences=S)
        l, i = torch.randn(T, 16, device="cuda"), torch.zeros(T, 2, dtype=torch.int32, device="cuda")
        o = torch.linspace(0, T, S + 1, device="cuda").int()
        m = torch.zeros(T, dtype=torch.uint8, device="cuda")
        balance.forward(b, l, i, seq_offsets=o, mask=m, z_coef=1.0)
        d = torch.ones(T, 16, device="cuda")
        balance.backward(b, l, d, seq_offsets=o, mask=m, z_coef=1.0, accumulate=False)
        balance.check(b)
        for t in (b.losses, b.counts, b.prob_mean, b.seq_tokens, d):
            assert torch.count_nonzero(t) == 0


def test_bad_contents_are_reported():
    """Indices and offsets out of range: skipped or clamped on the device, and told in the status word."""
    from dropless_mixture_experts_warp_gb300 import balance, binding as B
    l, idx, offsets, _ = case(300, 16, 2, 3, False)
    for change in ("index", "negative index", "order", "end", "start", "far"):
        j, o = idx.copy(), offsets.copy()
        if change == "index":
            j[5, 1] = 16
        elif change == "negative index":
            j[5, 1] = -1
        elif change == "order":
            o[1], o[2] = 200, 100
        elif change == "end":
            o[3] = 299
        elif change == "start":
            o[0] = 1
        else:
            o[3] = 1 << 30
        b = balance.allocate(300, 16, 2, sequences=3)
        dl, di, do = cuda(l, j, o)
        balance.forward(b, dl, di, seq_offsets=do)
        with pytest.raises(B.MoeError) as e:
            balance.check(b)
        assert e.value.status == 7, change
        if "index" in change:
            assert int(b.counts.sum()) == 599


def test_side_stream_and_graph():
    from dropless_mixture_experts_warp_gb300 import balance
    l, idx, offsets, mask = cuda(*case(900, 128, 8, 4, True))
    b = balance.allocate(900, 128, 8, sequences=4)
    kw = dict(seq_offsets=offsets, mask=mask, coef=COEF, z_coef=Z)
    balance.forward(b, l, idx, **kw)
    d = balance.backward(b, l, torch.zeros_like(l), **kw)
    want = [t.clone() for t in (b.losses, b.counts, b.prob_mean, d)]
    other = balance.allocate(900, 128, 8, sequences=4)
    side, d2 = torch.cuda.Stream(), torch.zeros_like(l)
    side.wait_stream(torch.cuda.current_stream())
    balance.forward(other, l, idx, stream=side, **kw)
    balance.backward(other, l, d2, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, (other.losses, other.counts, other.prob_mean, d2)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        balance.forward(b, l, idx, **kw)
        balance.backward(b, l, d, accumulate=False, **kw)
    for t in (b.losses, b.counts, b.prob_mean):
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, (b.losses, b.counts, b.prob_mean, d)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S,masked", [(14000, 256, 8, 6, True), (6500, 1000, 4, 1, False), (4000, 301, 8, 3, True),
                                            (90000, 16, 2, 600, True), (12000, 512, 8, 2, False), (25000, 127, 6, 30, True)])
def test_many_tokens(T, E, k, S, masked, score):
    """Several tokens a group and several groups a block's part; more sequences than the table in shared memory."""
    run(*case(T, E, k, S, masked), score, k)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S,masked", [(9001, 7, 7, 1, True), (5003, 15, 12, 3, True), (16, 16, 16, 2, False),
                                            (6001, 18, 9, 1, False), (5501, 33, 10, 4, True), (5002, 66, 5, 1, True),
                                            (4001, 131, 17, 2, False), (2501, 258, 8, 1, True), (9000, 32, 20, 3, True)])
def test_each_number_of_lanes(T, E, k, S, masked, score):
    """Widths that are no multiple of four at each group size, and more choices than a group reads ahead."""
    run(*case(T, E, k, S, masked, 1), score, k)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_the_gradient_takes_the_forwards_coefficients(score):
    """backward() without coefficients is the gradient of the losses that forward() gave; others hold for one call."""
    from dropless_mixture_experts_warp_gb300 import balance
    l, idx, offsets, mask = case(300, 24, 3, 4, True, 2)
    b = balance.allocate(300, 24, 3, score=score, sequences=4)
    dl, di, do, dm = cuda(l, idx, offsets, mask)
    at = dict(seq_offsets=do, mask=dm)
    balance.forward(b, dl, di, coef=COEF, z_coef=Z, **at)
    ref = oa.balance_fwd(l.astype(np.float64), idx, offsets, mask, 3, score, COEF, Z)

    def bound(wanted_coef, wanted_z, **given):
        d, m = oa.balance_bwd(l.astype(np.float64), offsets, mask, ref["counts"], ref["seq_tokens"], 3, score,
                              wanted_coef, wanted_z)
        out = balance.backward(b, dl, torch.zeros(300, 24, device="cuda"), accumulate=False, **at, **given)
        check(str(given), out, (d, m), "fp32", 2 * ROW)

    bound(COEF, Z)
    bound(2.0, Z, coef=2.0)
    bound(COEF, 0.0, z_coef=0.0)
    bound(3.0, 0.125, coef=3.0, z_coef=0.125)
    bound(COEF, Z)


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_written_just_before_and_on_another_stream(captured):
    """The kernels come up while what precedes them runs, and the forward's second one reads the offsets before it
    waits: logits, choices, offsets and mask written by a slow kernel or a copy, of the call's stream or of another
    that it waits for, count all the same, and what follows may overwrite them."""
    from dropless_mixture_experts_warp_gb300 import balance
    T, E, k, S = 6000, 64, 6, 5
    l, idx, offsets, mask = cuda(*case(T, E, k, S, True, 3))
    b = balance.allocate(T, E, k, sequences=S)
    outs = lambda: [b.losses, b.counts, b.prob_mean, b.seq_tokens]  # noqa: E731
    balance.forward(b, l, idx, seq_offsets=offsets, mask=mask, coef=COEF, z_coef=Z)
    want = [t.clone() for t in outs()]
    want.append(balance.backward(b, l, torch.zeros_like(l), seq_offsets=offsets, mask=mask).clone())
    balance.check(b)
    # what stands in the arrays before: other numbers, all of them in range
    spare = [torch.zeros_like(l), torch.zeros_like(idx), torch.linspace(0, T, S + 1, device="cuda").int(), torch.ones_like(mask)]
    src, got = [t.clone() for t in spare], [torch.zeros_like(t) for t in want]
    side = torch.cuda.Stream()

    def fill():
        torch.cuda._sleep(200_000)
        for dst, t in zip(src, (l, idx, offsets, mask)):
            dst.copy_(t)

    def spoil():
        for dst, t in zip(src, spare):
            dst.copy_(t)

    def work():
        here = torch.cuda.current_stream()
        d, at = got[-1], dict(seq_offsets=src[2], mask=src[3])
        fill()
        balance.forward(b, src[0], src[1], coef=COEF, z_coef=Z, **at)
        spoil()
        for t, o in zip(got, outs()):
            t.copy_(o)
        d.zero_()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            fill()
        here.wait_stream(side)
        balance.backward(b, src[0], d, **at)
        spoil()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    s.synchronize()
    if captured:
        for t in got:
            t.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            work()
        torch.cuda.synchronize()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
