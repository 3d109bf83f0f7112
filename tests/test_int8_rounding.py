"""The arithmetic by which 16-bit rows are quantised without comparing products:
127 / amax rounded up to FP32, one exact product rounded to a whole number. Every
pair of significands, at every distance in powers of two that gives a code."""
import numpy as np
import pytest


@pytest.mark.parametrize("bits", [8, 11])
def test_codes_from_the_factor_rounded_up(bits):
    A = np.arange(2 ** (bits - 1), 2 ** bits, dtype=np.int64)[:, None]
    X = A.T
    factor = (127.0 / A).astype(np.float32)
    # FP64 holds factor * A exactly: 24 + 11 bits
    factor = np.where(factor.astype(np.float64) * A < 127.0, np.nextafter(factor, np.float32(np.inf)), factor)
    exact = factor.astype(np.float64) * A == 127.0
    wrong = np.zeros(len(A), dtype=bool)
    for j in range(10):
        got = np.rint(factor.astype(np.float64) * (X * 2.0 ** -j))        # exact product, to nearest even
        num, den = 254 * X, 2 * A * 2 ** j                                # q = num / den
        k, rest = num // den, 2 * (num % den)
        want = k + ((rest > den) | ((rest == den) & (k % 2 == 1)))
        wrong |= ((got != want) & (X <= A * 2 ** j)).any(axis=1)
    # rows that the kernel compares: 127 divides the significand and the factor is not exact
    compared = ((A % 127 == 0) & ~exact)[:, 0]
    assert not (wrong & ~compared).any()
    if bits == 8:
        assert not compared.any()
