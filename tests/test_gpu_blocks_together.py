"""The 8-bit products, the layer and Muon as they are used together: training steps, graphs, streams, repeats, large sizes."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu
from oracle import blocks as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def stack(prec="fp8-block", optimizer="muon", **kw):
    from dropless_mixture_experts_warp_gb300 import train
    return train.Stack(300, 256, 128, 8, 2, prec=prec, optimizer=optimizer, **kw)


def inputs(model):
    g = torch.Generator("cuda").manual_seed(3)
    h = torch.randn(300, 256, device="cuda", generator=g).to(model.stream)
    return h, torch.randn(300, 256, device="cuda", generator=g)


def one_step(model, h, target, t):
    x = model.forward(h)
    model.backward((2 * (x.float() - target) / target.numel()).bfloat16())
    grads = [b.dw_gu.clone() for b in model.bufs] + [b.dw_d.clone() for b in model.bufs]
    model.update(t, lr=1e-3)
    return grads


def test_training_steps():
    """Three steps: gradients of the experts are the columns' forms' products, weights move by Muon's formula, copies are
    the weights rounded, the rest goes through AdamW."""
    model = stack()
    h, target = inputs(model)
    for t in range(1, 4):
        w0 = [w.double().cpu().numpy() for w in model.matrices.weights]
        m0 = [m.double().cpu().numpy() for m in model.matrices.m]
        gate0 = model.blocks[0]["gate"].clone()
        one_step(model, h, target, t)
        model.check()
        for b in model.bufs:
            off = b.row_offsets.tolist()
            n = off[-1]
            cols = lambda r: ob.rows_values(r.codes_t[:, :n].cpu(), r.scales_t[: n // 128].cpu().numpy()).T  # noqa: E731
            for got, dy, x in ((b.dw_gu, b.q.dgu, b.q.x), (b.dw_d, b.q.dy, b.q.h)):
                ref, mag = ob.weight_grad(cols(dy), cols(x), off)
                bound = ob.BF16_HALF * np.abs(ref) + 4 * (n + 2) * ob.U32 * mag + 1e-37
                assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound)
        p = model.matrices
        for i, w in enumerate(p.weights):
            rows, cols_ = w.shape[-2:]
            flat = lambda a: np.asarray(a).reshape(-1, rows, cols_)  # noqa: E731
            g = flat(p.grads[i].double().cpu().numpy())
            new = flat(w.double().cpu().numpy())
            for k in range(0, len(g), 3):
                ref, _, o = ob.muon_step(flat(w0[i])[k], flat(m0[i])[k], g[k], 1e-3, 0.95, 0.1, 0.2)
                u = g[k] + 0.95 * (0.95 * flat(m0[i])[k] + g[k])
                low = ob.newton_schulz_rounded(u)
                e = np.linalg.norm((low.T if rows > cols_ else low) - o)
                size = 1e-3 * 0.2 * np.sqrt(max(rows, cols_))
                assert np.linalg.norm(new[k] - ref) <= size * (1.5 * e + 2.0 ** -11 * np.linalg.norm(o)) + 4 * ob.U32 * np.linalg.norm(np.abs(ref) + size * np.abs(o))
            if p.copies[i] is not None:
                assert torch.equal(p.copies[i], w.bfloat16())
        assert not torch.equal(gate0, model.blocks[0]["gate"])


@pytest.mark.parametrize("prec,optimizer", [("fp8-block", "adamw"), ("bf16", "muon"), ("mxfp8", "muon")])
def test_other_pairs_run(prec, optimizer):
    model = stack(prec, optimizer)
    h, target = inputs(model)
    for t in (1, 2):
        one_step(model, h, target, t)
    model.check()
    assert all(torch.isfinite(w).all() for b in model.blocks for w in b.values())
    with pytest.raises(ValueError):
        stack(optimizer="sgd")


def test_repeats_give_the_same_bits():
    a, b = [], []
    for out in (a, b):
        model = stack()
        h, target = inputs(model)
        out += one_step(model, h, target, 1) + one_step(model, h, target, 2) + [w.clone() for w in model.matrices.weights]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def serving(T, rng, d=512, f=256, E=16, k=4):
    from dropless_mixture_experts_warp_gb300 import fp8, layer
    b = layer.allocate(layer.dims_of(T, d, f, E, k, prec="fp8-block"), train=False)
    cuda = lambda *s: torch.from_numpy(rng.standard_normal(s) * 0.05).bfloat16().cuda()  # noqa: E731
    gu = fp8.quantize_weights(fp8.allocate_weights(E, 2 * f, d), cuda(E, 2 * f, d))
    down = fp8.quantize_weights(fp8.allocate_weights(E, d, f), cuda(E, d, f))
    layer.use_weights(b, gu, down)
    x = torch.from_numpy(rng.standard_normal((T, d))).bfloat16().cuda()
    return b, x, torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()


@pytest.mark.parametrize("T", [1, 3, 64])
def test_captured_serving(T):
    """A captured forward, replayed on new inputs and routing, gives an eager one's bits."""
    from dropless_mixture_experts_warp_gb300 import layer
    b, x, logits = serving(T, np.random.default_rng(T))
    layer.forward(b, x, logits, None, None, weights_cached=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(b, x, logits, None, None, weights_cached=True)
    for seed in (1, 2):
        x.normal_(generator=torch.Generator("cuda").manual_seed(seed))
        logits.normal_(generator=torch.Generator("cuda").manual_seed(10 + seed))
        graph.replay()
        got = b.y.clone()
        assert torch.equal(got, layer.forward(b, x, logits, None, None, weights_cached=True))
    layer.check(b)


def test_inputs_written_just_before_on_another_stream():
    """Work on a side stream, its inputs written there by the kernel before it (early launches wait for it)."""
    from dropless_mixture_experts_warp_gb300 import fp8
    side = torch.cuda.Stream()
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((700, 1024))).bfloat16().cuda()
    w = fp8.quantize_weights(fp8.allocate_weights(1, 384, 1024), torch.from_numpy(rng.standard_normal((1, 384, 1024))).bfloat16().cuda())
    a, out = fp8.allocate_rows(700, 1024), torch.empty(700, 384, dtype=torch.bfloat16, device="cuda")
    want = fp8.matmul(fp8.quantize(a, x), w, out).clone()
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    for _ in range(20):
        y.zero_()
        a.codes.view(torch.uint8).zero_()
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mul(x, 1, out=y)
            fp8.quantize(a, y)
            fp8.matmul(a, w, out)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want)
    fp8.matmul(a, w, out.zero_(), stream=side)                  # a stream by argument
    side.synchronize()
    assert torch.equal(out, want)
    fp8.check(a)


def test_offsets_past_32_bits():
    """More than 2^31 elements in the quantiser and the product's rows; the last rows are right."""
    from dropless_mixture_experts_warp_gb300 import fp8
    R, C = 300_013, 7168
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(5))
    a = fp8.quantize(fp8.allocate_rows(R, C, both=True), x)
    w = fp8.quantize_weights(fp8.allocate_weights(1, 16, C), torch.randn(1, 16, C, device="cuda").bfloat16())
    out = fp8.matmul(a, w, torch.empty(R, 16, dtype=torch.bfloat16, device="cuda"))
    fp8.check(a)
    lo = R // 128 * 128
    tail = x[lo:].float().cpu().numpy()
    codes, scales = ob.quantize_rows(tail)
    assert torch.equal(a.codes[lo:].view(torch.uint8).cpu(), codes.view(torch.uint8)) and np.array_equal(a.scales[:, lo:].cpu().numpy(), scales)
    codes_t, scales_t = ob.quantize_columns(tail)
    assert torch.equal(a.codes_t[:, lo:].contiguous().view(torch.uint8).cpu(), codes_t.view(torch.uint8))
    assert np.array_equal(a.scales_t[-1:].cpu().numpy(), scales_t)
    ref, mag = ob.product(ob.rows_values(codes, scales), ob.weights_values(w.codes.cpu(), w.scales.cpu().numpy()))
    assert np.all(np.abs(out[lo:].double().cpu().numpy() - ref) <= ob.BF16_HALF * np.abs(ref) + 4 * (C + 2) * ob.U32 * mag)


def test_many_experts_and_wide_rows():
    """The limits: 1024 experts, most of them empty; one row each in some."""
    from dropless_mixture_experts_warp_gb300 import fp8
    rng = np.random.default_rng(6)
    E, N, K = 1024, 144, 272
    counts = np.zeros(E, int)
    counts[[0, 5, 511, 1000, 1023]] = [1, 300, 128, 2, 7]
    off = np.concatenate([[0], np.cumsum(-(-counts // 128) * 128)])
    x = rng.standard_normal((off[-1], K)).astype(np.float32)
    codes, scales = ob.quantize_rows(x)
    wc = torch.from_numpy((rng.standard_normal((E, N, K)) * 50).astype(np.float32)).to(ob.E4M3)
    ws = (rng.random((E, 2, 3)) * 1e-3).astype(np.float32)
    a = fp8.rows_of(codes.cuda(), torch.from_numpy(scales).cuda())
    o = torch.from_numpy(off.astype(np.int32)).cuda()
    out = fp8.matmul(a, fp8.weights_of(wc.cuda(), torch.from_numpy(ws).cuda()), torch.empty(off[-1], N, dtype=torch.bfloat16, device="cuda"), offsets=o)
    ref, mag = ob.product(ob.rows_values(codes, scales), ob.weights_values(wc, ws), off)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= ob.BF16_HALF * np.abs(ref) + 4 * (K + 2) * ob.U32 * mag + 1e-37)
    cc, cs = ob.quantize_columns(x)
    t = fp8.rows_of(codes_t=cc.cuda(), scales_t=torch.from_numpy(cs).cuda())
    g = fp8.weight_grad(t, t, torch.full((E, K, K), 7.0, dtype=torch.bfloat16, device="cuda"), offsets=o)
    fp8.check(t)
    v = ob.rows_values(cc, cs).T
    ref, mag = ob.weight_grad(v, v, off)
    assert np.all(np.abs(g.double().cpu().numpy() - ref) <= ob.BF16_HALF * np.abs(ref) + 4 * 400 * ob.U32 * mag + 1e-37)


def test_two_streams_at_once():
    """Two sets of buffers on two streams at once, called and as graphs, give what each gives alone."""
    from dropless_mixture_experts_warp_gb300 import fp8, muon
    g = torch.Generator("cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731

    def chain(R, N, K, E):
        x, dy, w16 = r(R, K), r(R, N), r(E, N, K)
        off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (R // E // 128 * 128)
        a, b, w = fp8.allocate_rows(R, K, both=True), fp8.allocate_rows(R, N, both=True), fp8.allocate_weights(E, N, K, both=True)
        out, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w16)
        o, ws = torch.empty_like(dw), muon.workspace([dw.shape])

        def run(s=None):
            fp8.quantize(a, x, stream=s), fp8.quantize(b, dy, stream=s), fp8.quantize_weights(w, w16, stream=s)
            fp8.matmul(a, w, out, off, stream=s)
            fp8.matmul(b, w, dx, off, transposed=True, stream=s)
            fp8.weight_grad(b, a, dw, off, stream=s)
            muon.orthogonalize([dw], [o], ws, stream=s)
            return out, dx, dw, o, a, b, ws
        return run

    chains = [chain(4096, 1536, 768, 8), chain(1000, 528, 2064, 3)]
    alone = [[t.clone() for t in run()[:4]] for run in chains]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    graphs = []
    for run, s in zip(chains, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            run(s.cuda_stream)

    def compare(outs):
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for got, want in zip(outs, alone) for x, y in zip(got, want))

    for _ in range(20):
        outs = [run(s.cuda_stream) for run, s in zip(chains, streams)]
    compare(outs)
    for got in outs:
        for t in got[:4]:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    compare(outs)
    for got in outs:
        fp8.check(got[4]), fp8.check(got[5]), muon.check(got[6])
