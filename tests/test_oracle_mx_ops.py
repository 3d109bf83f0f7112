"""The MXFP4 operators' oracle, pinned: quantisation by brute force over every
pair of neighbouring values and by its own properties, scale tiles by the
index formula, routing and experts by worked cases."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mxfp4_ops_oracle as Q
from oracle.mxfp4_oracle import e2m1_decode

MAGS = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]


def brute_code(v: Fraction) -> int:
    """Nearest E2M1 code of an exact rational, ties to even, saturating."""
    a = abs(v)
    best = min(range(8), key=lambda c: (abs(a - MAGS[c]), c % 2))
    return best | (8 if v < 0 else 0)


def block(values):
    b = np.zeros(32)
    b[:len(values)] = values
    return b


def test_every_boundary_of_the_grid():
    # amax = 4 fixes e = 127; every multiple of 1/64 up to 8 is compared exactly
    for lead in (4.0, 7.75):
        for first in range(0, 64 * 8, 31):
            vals = [lead] + [(first + i) / 64.0 * (-1) ** i for i in range(31) if (first + i) / 64.0 < 8]
            c, e = Q.quantize_blocks(block(vals))
            assert e == 127
            for got, v in zip(c, vals):
                want = brute_code(Fraction(v))
                assert e2m1_decode(got) == e2m1_decode(want), (v, got, want)


@pytest.mark.parametrize("v,code", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (6.5, 7)])
def test_ties_go_to_the_even_code(v, code):
    c, _ = Q.quantize_blocks(block([7.0, v, -v]))
    assert c[1] == code and c[2] == code + 8


@pytest.mark.parametrize("p", [-140, -126, -125, -60, 0, 1, 60, 127])
def test_exponent_byte(p):
    for m in (1.0, 1.5, 2.0 - 2.0 ** -20):
        _, e = Q.quantize_blocks(block([np.ldexp(m, p), 0.0]))
        assert e == max(p - 2 + 127, 0)


def test_zero_and_non_finite_blocks():
    c, e = Q.quantize_blocks(np.zeros(32))
    assert e == 0 and not c.any()
    for bad in (np.inf, -np.inf, np.nan):
        c, e = Q.quantize_blocks(block([1.0, bad, 3.0]))
        assert e == 255 and not c.any()


def test_idempotent_on_its_own_values():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((7, 96)) * np.exp(rng.standard_normal((7, 1)) * 5)
    c, e = Q.quantize(x, 1)
    v = Q.values(c, e, 1)
    c2, e2 = Q.quantize(v, 1)
    assert np.array_equal(Q.values(c2, e2, 1), v)
    # and along the other axis
    c0, e0 = Q.quantize(x.T, 0)
    assert np.array_equal(c0.T, c) and np.array_equal(e0.T, e)


def test_error_is_at_most_half_a_step():
    rng = np.random.default_rng(4)
    v = rng.standard_normal((50, 32))
    c, e = Q.quantize_blocks(v)
    scale = np.ldexp(1.0, e.astype(int) - 127)[:, None]
    # steps of the grid are at most 2 below 6; what lies in (6, 8) loses less than 2
    assert np.all(np.abs(e2m1_decode(c) * scale - v) <= np.where(np.abs(v) / scale > 6, 2.0, 1.0) * scale)


def test_tile_index_formula():
    e = np.arange(130 * 9, dtype=np.int64).reshape(130, 9) % 251
    t = Q.tile_scales(e.astype(np.uint8)).reshape(-1)
    groups = 3
    for r in (0, 1, 31, 32, 127, 128, 129):
        for b in (0, 3, 4, 8):
            at = ((r // 128) * groups + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
            assert t[at] == e[r, b]


def test_route_ties_and_weights():
    idx, w = Q.route(np.array([[1.0, 3.0, 3.0, 2.0]]), 2, False)
    assert idx.tolist() == [[1, 2]]
    z = np.exp([1.0, 3.0, 3.0, 2.0])
    assert np.allclose(w, [[z[1] / z.sum()] * 2])
    _, w = Q.route(np.array([[1.0, 3.0, 3.0, 2.0]]), 2, True)
    assert np.allclose(w, [[0.5, 0.5]])


def test_one_expert_is_a_plain_gated_mlp():
    rng = np.random.default_rng(5)
    H, inner = 32, 32
    x = rng.standard_normal((3, H))
    w13 = rng.integers(0, 16, size=(1, H, 2 * inner)).astype(np.uint8)
    w2 = rng.integers(0, 16, size=(1, inner, H)).astype(np.uint8)
    e13 = np.full((1, 1, 2 * inner), 124, dtype=np.uint8)
    e2 = np.full((1, 1, H), 125, dtype=np.uint8)
    y = Q.experts(x, np.zeros((1, H)), w13, e13, w2, e2, 1, True)
    a = x @ (e2m1_decode(w13[0]) / 8)
    h = a[:, :inner] / (1 + np.exp(-a[:, :inner])) * a[:, inner:]
    assert np.allclose(y, h @ (e2m1_decode(w2[0]) / 4))


def test_byte_counts():
    from weight_only_int4_gb300.accounting import mx_matmul_bytes, mx_moe_bytes, mx_quantize_bytes
    assert mx_quantize_bytes(64, 2) == 64 * 2 + 32 + 2
    assert mx_matmul_bytes(2, 8, 64, 4) == 2 * 34 + 8 * 34 + 2 * 8 * 4
    # one token reads its k experts; with k = E every expert is read
    assert mx_moe_bytes(1, 8, 2, 64, 32) == 2 * 3 * 64 * 32 * 17 // 32 + 8 * 64 * 2 + 2 * 64 * 2
    assert mx_moe_bytes(5, 4, 4, 64, 32) == 4 * 3 * 64 * 32 * 17 // 32 + 4 * 64 * 2 + 2 * 5 * 64 * 2
