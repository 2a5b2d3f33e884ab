"""The float64 forms of the operators around the layer: gradients against differences (CPU)."""
import numpy as np
import pytest

from oracle import around as oa

EPS = 1e-6


def differences(f, x, g, step=1e-6):
    """d sum(g * f(x)) / dx by central differences, element by element."""
    out = np.empty_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + step
        hi = (g * f()).sum()
        x[i] = keep - step
        lo = (g * f()).sum()
        x[i] = keep
        out[i] = (hi - lo) / (2 * step)
    return out


# a central difference of a smooth function of size ~1: step^2 for the cut, 2^-53 / step for the rounding of a
# sum of some tens of terms; both under 1e-8, asked for at 1e-6
TOL = 1e-6


def test_norm_gradients_are_the_differences():
    rng = np.random.default_rng(1)
    h, w, g, add = (rng.standard_normal(s) for s in ((3, 8), (8,), (3, 8), (3, 8)))
    got = oa.norm_bwd(g, h, w, EPS, 1.0, add)
    f = lambda: oa.norm_fwd(h, w, EPS, 1.0)  # noqa: E731
    assert abs(got["dh"][0] - add - differences(f, h, g)).max() < TOL
    assert abs(got["dw"][0] - differences(f, w, g)).max() < TOL


@pytest.mark.parametrize("kind,sigmoid", [("none", False), ("channel", False), ("channel", True), ("token", True)])
@pytest.mark.parametrize("post", [True, False])
def test_merge_gradients_are_the_differences(kind, sigmoid, post):
    rng = np.random.default_rng(2)
    T, d = 3, 8
    h, y, g, gx = (rng.standard_normal((T, d)) for _ in range(4))
    w_post = rng.standard_normal(d) if post else None
    w_next = rng.standard_normal(d)
    gate = None if kind == "none" else rng.standard_normal(d if kind == "channel" else T)
    opt = dict(eps=EPS, kind=kind, sigmoid=sigmoid, offset=0.5, alpha=0.7, beta=1.3)
    h_out = oa.merge_fwd(h, y, w_post, gate, w_next, **opt)["h_out"][0]
    got = oa.merge_bwd(g, gx, h_out, y, w_post, gate, w_next, **opt)

    def both():
        r = oa.merge_fwd(h, y, w_post, gate, w_next, **opt)
        return np.stack([r["h_out"][0], r["x"][0]])

    gg = np.stack([g, gx])
    wanted = {"dh": h, "dy": y, "dw_next": w_next}
    if post:
        wanted["dw_post"] = w_post
    if gate is not None:
        wanted["dgate"] = gate
    assert set(got) == set(wanted)
    for name, x in wanted.items():
        assert abs(got[name][0] - differences(both, x, gg)).max() < TOL, name


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_is_the_difference(score):
    rng = np.random.default_rng(3)
    T, E, k = 12, 6, 2
    l = rng.standard_normal((T, E))
    idx = np.argsort(-l, axis=1)[:, :k].copy()
    mask = np.ones(T, np.uint8)
    mask[[4, 11]] = 0
    offsets = np.array([0, 5, 5, 12])
    fwd = oa.balance_fwd(l, idx, offsets, mask, k, score, 0.7, 0.3)
    assert fwd["seq_tokens"].tolist() == [4, 0, 6] and fwd["counts"].sum() == k * 10
    grad = (1.5, 0.5)
    got, _ = oa.balance_bwd(l, offsets, mask, fwd["counts"], fwd["seq_tokens"], k, score, 0.7, 0.3, grad)
    f = lambda: oa.balance_fwd(l, idx, offsets, mask, k, score, 0.7, 0.3)["losses"]  # noqa: E731
    assert abs(got - differences(f, l, np.array(grad))).max() < TOL


def test_balance_of_an_even_router_is_the_coefficient():
    """Uniform probabilities: sum f P = (1 / E) sum f = 1, whatever the counts."""
    l = np.zeros((8, 4))
    idx = np.arange(8)[:, None] % 4
    fwd = oa.balance_fwd(l, idx, np.array([0, 8]), None, 1, "softmax", 0.25, 1.0)
    assert np.allclose(fwd["losses"], [0.25, np.log(4.0) ** 2])


@pytest.mark.parametrize("top,power", [(127, 2), (255, 4)])
def test_codes_have_the_value_as_their_mean(top, power):
    """Over 4000 draws the mean of the decoded value is within 5 standard errors (at most half a code's width each)."""
    rng = np.random.default_rng(4)
    x = rng.random(128) ** 3 * 2.5e-4
    if power == 2:
        x *= rng.choice([-1.0, 1.0], 128)
    s = oa.block_scales(x)
    assert s[0] == abs(x).max()
    got = np.stack([oa.decode(oa.encode(x, s, oa.adamw_draws(seed, 3, 1, 128)[power // 4], top, power)[0], s, top, power)
                    for seed in range(4000)])
    k = (abs(x) / s[0]) ** (1 / power) * top
    width = s[0] * (((np.floor(k) + 1) / top) ** power - (np.floor(k) / top) ** power)
    # codes of v below 1 are raised to 1: only shares above that are unbiased
    fair = k >= 1 if power == 4 else k >= 0
    assert fair.sum() > 100
    assert np.all(abs(got.mean(axis=0) - x)[fair] <= 5 * 0.5 * width[fair] / np.sqrt(4000) + 1e-12 * s[0])
    assert np.all(abs(got - x)[:, fair] <= width[fair] * (1 + 1e-9))
    if power == 4:
        assert np.all(got > 0)
    assert oa.encode(np.zeros(128), np.zeros(1), np.full(128, 0.5), top, power)[0].max() == 0


def test_draws_are_even_and_do_not_follow_each_other():
    """The 16-bit draws of neighbouring elements, steps, tensors and seeds: means, variances and correlations within
    5 standard errors."""
    n = 1 << 16
    sets = [oa.adamw_draws(*a, n) for a in [(0, 1, 0), (0, 2, 0), (0, 1, 1), (1, 1, 0)]] + [oa.adamw_draws(0, 1, 0, n, 1 << 32)]
    flat = [u for pair in sets for u in pair]
    for u in flat:
        assert abs(u.mean() - 0.5) < 5 * (1 / 12) ** 0.5 / n ** 0.5
        assert abs(u.var() - 1 / 12) < 5 * (1 / 180) ** 0.5 / n ** 0.5
        assert abs(np.corrcoef(u[:-1], u[1:])[0, 1]) < 5 / n ** 0.5
    for i, a in enumerate(flat):
        for b in flat[:i]:
            assert abs(np.corrcoef(a, b)[0, 1]) < 5 / n ** 0.5


def test_8_bit_moments_follow_the_32_bit_ones():
    """A moment that moves by less than a code's width a step still decays: after 2000 steps of gradients 30 times
    smaller the mean over 512 elements is within 10% (each element's noise is under half a code: 1/15 of v at code
    60, and 512 of them average)."""
    rng = np.random.default_rng(6)
    n, beta2 = 512, 0.999
    v = np.full(n, 1.0)
    s, code = np.ones(n // 128), np.full(n, 255)
    for t in range(1, 2001):
        g2 = (rng.standard_normal(n) / 30) ** 2
        v = beta2 * v + (1 - beta2) * g2
        new = beta2 * oa.decode(code, s, 255, 4) + (1 - beta2) * g2
        s = oa.block_scales(new)
        code = oa.encode(new, s, oa.adamw_draws(9, t, 0, n)[1], 255, 4)[0]
    assert v.mean() < 0.2
    assert abs(oa.decode(code, s, 255, 4).mean() / v.mean() - 1) < 0.1
