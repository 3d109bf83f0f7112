"""CPU FP64 oracle for the int8 operators: rows quantised to int8, the product of
int8 operands, the step between two blocks.

TEST INFRASTRUCTURE ONLY, as the other oracles: the product never calls it and
shares no code with it.

    quantise   scale = RN_f32(amax / 127), code = the whole number nearest to
               127 v / amax, ties to even; a row of zeros: scale 0, codes 0; a
               row with an infinity or a NaN: scale NaN, codes 0
    product    y[m, n] = (sum_k a[m, k] b[n, k]) * sa[m] * sb[n]
    norm       u = h rsqrt(mean(h^2) + eps) after, r' = r + scale gate u,
               y = r' rsqrt(mean(r'^2) + eps) weight

Parity status of each function (pins in the tests):
  quantize_rows ....... pinned (exact rational brute force)
  product ............. pinned (Python integers)
  block_norm .......... pinned (one row in exact rationals and square roots)
"""
from __future__ import annotations

import numpy as np


def quantize_rows(x: np.ndarray):
    """x [R, K] FP64 holding exact values of the input type -> (codes int8 [R, K], scale float32 [R])."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x).all(axis=1)
    v = np.where(fine[:, None], x, 0.0)
    amax = np.abs(v).max(axis=1)
    safe = np.where(amax > 0, amax, 1.0)
    # inputs have at most 24 bits, so the quotient is at least 2^-33 of itself away from a half it does not
    # equal, and its rounding to 53 bits changes no decision
    codes = np.rint(127.0 * v / safe[:, None]).astype(np.int8)
    scale = (amax / 127.0).astype(np.float32)
    return codes, np.where(fine, scale, np.float32(np.nan)).astype(np.float32)


def product(a, sa, b, sb) -> np.ndarray:
    acc = np.asarray(a, dtype=np.int64) @ np.asarray(b, dtype=np.int64).T
    return acc.astype(np.float64) * np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64)


def block_norm(residual, weight, h=None, after=None, gate=None, scale=1.0, eps=1e-6):
    """(r', y), y None without weight. gate broadcasts against [T, H]."""
    r = np.asarray(residual, dtype=np.float64)
    if h is not None:
        u = np.asarray(h, dtype=np.float64)
        if after is not None:
            u = u / np.sqrt((u * u).mean(axis=1, keepdims=True) + eps) * np.asarray(after, np.float64)
        r = r + scale * (u if gate is None else u * np.asarray(gate, np.float64))
    if weight is None:
        return r, None
    return r, r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
