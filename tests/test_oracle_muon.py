"""Pins of oracle/blocks.py's forms of the orthogonalised update that its rounded arithmetics and floors have."""
import numpy as np
import pytest

from oracle import blocks as ob


@pytest.mark.parametrize("m,n", [(1, 1), (7, 40), (72, 131), (131, 72)])
def test_split_operands_are_as_good_as_22_bits(m, n):
    """Operands in two fp16 parts are a thousand times nearer than in one; what sums lose only adds to it."""
    x = np.random.default_rng(m).standard_normal((m, n))
    ref = ob.newton_schulz(x)
    turn = lambda r: r.T if m > n else r  # noqa: E731
    size = np.linalg.norm(ref)
    one = np.linalg.norm(turn(ob.newton_schulz_rounded(x)) - ref) / size
    two = np.linalg.norm(turn(ob.newton_schulz_split(x, step=0)) - ref) / size
    sums = np.linalg.norm(turn(ob.newton_schulz_split(x)) - ref) / size
    assert 1e-4 < one < 1e-2 and two < 4e-6 and two / 2 <= sums < 1e-3


def test_floor():
    """Over eps a matrix is divided by its norm, below by eps; the result then fades with it."""
    x = np.random.default_rng(0).standard_normal((20, 30))
    n = np.linalg.norm(x)
    assert np.array_equal(ob.newton_schulz(x, eps=n / 2), ob.newton_schulz(x))
    a, b, c = ob.COEFFICIENTS[0]
    y = x / (8 * n)
    want = a * y + b * y @ y.T @ y + c * y @ y.T @ y @ y.T @ y
    assert np.allclose(ob.newton_schulz(x, ob.COEFFICIENTS[:1], eps=8 * n), want, rtol=1e-12, atol=0)
    small = ob.newton_schulz(x * 2.0 ** -60, eps=n)
    assert 0 < np.linalg.norm(small) <= 3.4445 ** 5 * 2.0 ** -60
    assert not ob.newton_schulz(np.zeros((3, 4)), eps=1e-7).any()
