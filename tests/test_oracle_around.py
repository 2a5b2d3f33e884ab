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
