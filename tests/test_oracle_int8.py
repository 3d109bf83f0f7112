"""The int8 oracle against exact rationals and Python integers."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8_oracle as I8


def nearest_even(q: Fraction) -> int:
    low = math.floor(q)
    rest = q - low
    if rest != Fraction(1, 2):
        return low + (rest > Fraction(1, 2))
    return low + (low & 1)


@pytest.mark.parametrize("bits", [8, 11, 24])
def test_codes_against_rationals(bits):
    """Values of the input types' precisions; rows whose largest value makes ties common among them."""
    rng = np.random.default_rng(bits)
    tops = [1.0, 127.0, 254.0, 63.5, 1.9921875, 3.0, 1e30, 2.0 ** -60]
    for top in tops:
        m = rng.integers(0, 2 ** bits, 200) / 2.0 ** bits
        x = np.concatenate([[top], top * m * rng.choice([-1, 1], 200), [top / 2, -top / 2, 0.0]])
        x = np.ldexp(np.rint(np.ldexp(np.frexp(x)[0], bits)), np.frexp(x)[1] - bits)   # `bits` significant bits
        codes, scale = I8.quantize_rows(x[None])
        amax = max(abs(Fraction(float(v))) for v in x)
        assert [nearest_even(127 * Fraction(float(v)) / amax) for v in x] == codes[0].tolist()
        assert abs(Fraction(float(scale[0])) - amax / 127) <= amax / 127 * Fraction(1, 2 ** 24)


def test_special_rows():
    x = np.zeros((4, 16))
    x[1, 3], x[2, 4], x[3, 5] = np.inf, np.nan, 2.0 ** -149
    codes, scale = I8.quantize_rows(x)
    assert not codes[:3].any() and codes[3, 5] == 127
    assert scale[0] == 0 and np.isnan(scale[1:3]).all() and scale[3] == 0


def test_product_against_integers():
    rng = np.random.default_rng(1)
    a, b = rng.integers(-128, 128, (3, 48)), rng.integers(-128, 128, (5, 48))
    sa, sb = rng.random(3), rng.random(5)
    y = I8.product(a.astype(np.int8), sa, b.astype(np.int8), sb)
    for m in range(3):
        for n in range(5):
            want = sum(int(p) * int(q) for p, q in zip(a[m], b[n])) * sa[m] * sb[n]
            assert y[m, n] == pytest.approx(want, rel=1e-15)


def test_block_norm_row():
    r, h, after, gate, weight = ([Fraction(p, 7) for p in v] for v in
                                 ([1, -3, 5, 2], [4, 0, -2, 6], [7, 8, 6, 5], [1, 2, 3, 4], [9, 7, 5, 3]))
    eps, scale = Fraction(1, 1000), Fraction(3, 4)
    root = lambda v: math.sqrt(sum(x * x for x in v) / 4 + eps)  # noqa: E731
    u = [float(x) / root(h) * float(w) for x, w in zip(h, after)]
    want_r = [float(x) + float(scale * g) * v for x, g, v in zip(r, gate, u)]
    norm = math.sqrt(sum(x * x for x in want_r) / 4 + float(eps))
    arr = lambda v: np.array([[float(x) for x in v]])  # noqa: E731
    got_r, got_y = I8.block_norm(arr(r), arr(weight)[0], arr(h), arr(after)[0], arr(gate), float(scale), float(eps))
    assert got_r[0] == pytest.approx(want_r, rel=1e-14)
    assert got_y[0] == pytest.approx([x / norm * float(w) for x, w in zip(want_r, weight)], rel=1e-14)
    alone, none = I8.block_norm(arr(r), None, arr(h))
    assert none is None and alone[0] == pytest.approx([float(x + v) for x, v in zip(r, h)], rel=1e-15)
