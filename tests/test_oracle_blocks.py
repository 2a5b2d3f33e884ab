"""Pins of oracle/blocks.py: the codes by brute force, the orthogonal factor by singular values, gradients by differences."""
import numpy as np
import pytest
import torch

from oracle import blocks as ob


def test_codes_are_the_nearest_values():
    """Every code is a nearest E4M3 value of the quotient, ties to the even one; a block's largest value is code 448's."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((5, 300)) * 10.0 ** rng.integers(-6, 6, (5, 1))).bfloat16().float().numpy()
    codes, scales = ob.quantize_rows(x)
    grid = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(ob.E4M3).double().numpy()
    finite = np.unique(grid[np.isfinite(grid)])
    for r in range(5):
        for c in range(300):
            s = scales[c // 128, r]
            q = np.float32(x[r, c]) / s
            got = float(codes[r, c].float())
            assert abs(got - q) <= np.abs(finite - q).min() * (1 + 1e-12) + 1e-30
            near = finite[np.isclose(np.abs(finite - q), np.abs(finite - q).min(), rtol=1e-12, atol=0)]
            if len(near) == 2:
                byte = codes[r, c].view(torch.uint8).item()
                assert byte % 2 == 0
        for b in range(3):
            blk = slice(128 * b, min(300, 128 * (b + 1)))
            assert np.abs(codes[r, blk].float().numpy()).max() == 448.0
            assert scales[b, r] == np.float32(np.abs(x[r, blk]).max()) / np.float32(448)


def test_scales_of_nothing_and_of_tiny_blocks():
    assert ob.scale_of(np.zeros(1))[0] == np.float32(2.0 ** -64) / np.float32(448) == ob.scale_of(np.float32([1e-25]))[0]
    codes, _ = ob.quantize_rows(np.zeros((1, 16), np.float32))
    assert not codes.view(torch.uint8).any()
    codes, _ = ob.quantize_rows(-np.zeros((1, 16), np.float32))
    assert not codes.view(torch.uint8).any()


def test_forms_agree():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((256, 144)).astype(np.float32)
    c, s = ob.quantize_columns(x)
    r, t = ob.quantize_rows(np.ascontiguousarray(x.T))
    assert torch.equal(c.view(torch.uint8), r.view(torch.uint8)) and np.array_equal(s, t)
    w = rng.standard_normal((2, 200, 140)).astype(np.float32)
    codes, scales = ob.quantize_weights(w)
    off = np.abs(ob.weights_values(codes, scales) - w)
    step = scales.astype(np.float64).repeat(128, 1).repeat(128, 2)[:, :200, :140]
    assert np.all(off <= np.abs(w) * 2.0 ** -4 * (1 + 1e-6) + step * 2.0 ** -10)
    turned, st = ob.quantize_weights(np.ascontiguousarray(w.transpose(0, 2, 1)))
    assert torch.equal(turned.view(torch.uint8), codes.transpose(1, 2).contiguous().view(torch.uint8))
    assert np.array_equal(st, scales.transpose(0, 2, 1))


def test_products():
    rng = np.random.default_rng(2)
    a, w = rng.standard_normal((300, 20)), rng.standard_normal((3, 7, 20))
    off = [0, 128, 128, 256]
    y, mag = ob.product(a, w, off)
    owner = np.repeat([0, 2], 128)
    assert np.allclose(y[:256], np.einsum("rk,rnk->rn", a[:256], w[owner])) and np.isnan(y[256:]).all()
    assert np.all(mag[:256] >= np.abs(y[:256]) - 1e-12)
    g, _ = ob.weight_grad(a[:256, :5], a[:256, 5:], off)
    assert np.allclose(g[1], 0) and np.allclose(g[2], np.einsum("rn,rk->nk", a[128:256, :5], a[128:256, 5:]))


def test_swiglu_gradient_by_differences():
    rng = np.random.default_rng(3)
    g, u, w, dh = rng.standard_normal((4, 6)), rng.standard_normal((4, 6)), rng.random(4), rng.standard_normal((4, 6))
    dg, du, dw = ob.swiglu_bwd(g, u, w, dh)
    f = lambda g, u, w: (ob.swiglu(g, u, w) * dh).sum()  # noqa: E731
    e = 1e-6
    for i in range(4):
        d = np.zeros(4)
        d[i] = e
        assert abs((f(g, u, w + d) - f(g, u, w - d)) / (2 * e) - dw[i]) < 1e-7
        for j in range(6):
            d = np.zeros((4, 6))
            d[i, j] = e
            assert abs((f(g + d, u, w) - f(g - d, u, w)) / (2 * e) - dg[i, j]) < 1e-7
            assert abs((f(g, u + d, w) - f(g, u - d, w)) / (2 * e) - du[i, j]) < 1e-7


@pytest.mark.parametrize("m,n", [(5, 9), (9, 5), (6, 6), (1, 4)])
def test_newton_schulz_is_a_polynomial_of_the_singular_values(m, n):
    x = np.random.default_rng(m).standard_normal((m, n))
    u, s, v = np.linalg.svd(x / np.linalg.norm(x), full_matrices=False)
    for a, b, c in ob.COEFFICIENTS:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(ob.newton_schulz(x), (u * s) @ v, atol=1e-10)
    assert np.allclose(ob.newton_schulz(x * 1e-12), ob.newton_schulz(x), atol=1e-12)
    assert not ob.newton_schulz(np.zeros((m, n))).any()


def test_rounded_steps_are_the_same_polynomial():
    """Without its roundings' size the rounded form is newton_schulz: the terms taken off A and B cancel."""
    x = np.random.default_rng(7).standard_normal((48, 80))
    ref, low = ob.newton_schulz(x), ob.newton_schulz_rounded(x)
    assert np.linalg.norm(low - ref) < 4e-3 * np.linalg.norm(ref)
    tall = ob.newton_schulz_rounded(np.ascontiguousarray(x.T))
    assert np.array_equal(tall, low)
