"""CPU FP64 oracle for the MXFP4 operators: quantisation, the product of two
quantised operands, the mixture-of-experts layer.

TEST INFRASTRUCTURE ONLY, as the other oracles: the product never calls it and
shares no code with it.

    quantise   blocks of 32; with amax the largest magnitude of a block,
               e = max(floor(log2(amax)) - 2 + 127, 0), code = the E2M1 value
               nearest to v * 2^(127 - e), ties to the even code, 6 at most;
               a block with an infinity or a NaN: e = 255, codes 0
    product    y[m, n] = sum_k A[m, k] B[n, k] over decoded values
    experts    p = softmax(x R^T); the k largest logits, ties to the lower
               index; y = sum_e p_e ((silu(x W1_e) * (x W3_e)) W2_e), the p
               divided by their sum where renormalised

Parity status of each function (pins in the tests):
  quantize_blocks ..... pinned
  tile_scales ......... pinned
  route ............... pinned
  experts ............. pinned (against route and dequantize_mx one token at a time)
"""
from __future__ import annotations

import numpy as np

from oracle.mxfp4_oracle import MX_BLOCK, e2m1_decode, e8m0_decode
from oracle.w4a16_oracle import pack_cols, pack_rows


def quantize_blocks(v: np.ndarray):
    """v [..., 32] (FP64, exact values of the input type) -> codes uint8
    [..., 32], exponent bytes uint8 [...]."""
    v = np.asarray(v, dtype=np.float64)
    finite = np.isfinite(v).all(axis=-1)
    w = np.where(finite[..., None], v, 0.0)
    amax = np.abs(w).max(axis=-1)
    _, p = np.frexp(amax)                      # amax = m 2^p, m in [1/2, 1)
    e = np.where(amax > 0, np.maximum(p - 1 - 2 + 127, 0), 0)
    a = np.ldexp(np.abs(w), (127 - e)[..., None])
    mags = e2m1_decode(np.arange(8))
    dist = np.abs(a[..., None] - mags)         # exact: a and mags are short numbers
    best = dist.min(axis=-1, keepdims=True)
    tied = dist == best
    even = np.arange(8) % 2 == 0
    # the only nearest code, or the even one of two
    pick = np.where((tied & even).any(axis=-1), np.argmax(tied & even, axis=-1), np.argmax(tied, axis=-1))
    code = (pick | (np.signbit(w).astype(np.int64) << 3)).astype(np.uint8)
    code = np.where(finite[..., None], code, 0).astype(np.uint8)
    return code, np.where(finite, e, 255).astype(np.uint8)


def quantize(x: np.ndarray, dim: int):
    """x [R, C] FP64 -> (codes uint8 [R, C], bytes). Blocks along rows (dim 0,
    bytes [R/32, C]) or along columns (dim 1, bytes [R, C/32])."""
    x = np.asarray(x, dtype=np.float64)
    if dim == 0:
        c, e = quantize(x.T, 1)
        return np.ascontiguousarray(c.T), np.ascontiguousarray(e.T)
    R, C = x.shape
    if C % MX_BLOCK:
        raise ValueError("whole blocks only")
    c, e = quantize_blocks(x.reshape(R, C // MX_BLOCK, MX_BLOCK))
    return c.reshape(R, C), e


def words(codes: np.ndarray, dim: int) -> np.ndarray:
    """Packed int32 words, eight codes along `dim`."""
    return pack_rows(codes) if dim == 0 else pack_cols(codes)


def tile_scales(e: np.ndarray) -> np.ndarray:
    """[R, B] -> [ceil(R/128), ceil(B/4), 32, 4, 4], zero outside, one byte at a time."""
    R, B = e.shape
    out = np.zeros((-(-R // 128), -(-B // 4), 32, 4, 4), dtype=np.uint8)
    for r in range(R):
        for b in range(B):
            out[r // 128, b // 4, r % 32, (r // 32) % 4, b % 4] = e[r, b]
    return out


def values(codes: np.ndarray, e: np.ndarray, dim: int) -> np.ndarray:
    """FP64 values E2M1 * 2^(e - 127) (no rounding to a 16-bit type)."""
    s = e8m0_decode(e).repeat(MX_BLOCK, axis=dim)
    with np.errstate(invalid="ignore"):
        return e2m1_decode(codes) * s


def product(a_codes, a_e, b_codes, b_e) -> np.ndarray:
    """FP64 y [M, N] of row-layout operands [M, K], [N, K]."""
    with np.errstate(invalid="ignore"):
        return values(a_codes, a_e, 1) @ values(b_codes, b_e, 1).T


def route(logits: np.ndarray, k: int, renormalize: bool):
    """(indices, weights) [T, k], largest logit first, ties to the lower index."""
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    w = np.take_along_axis(p, idx, axis=1)
    if renormalize:
        w = w / w.sum(axis=1, keepdims=True)
    return idx, w


def experts(x, router, w13, e13, w2, e2, k: int, renormalize: bool) -> np.ndarray:
    """x [T, H], router [E, H] FP64; codes [E, H, 2I], [E, I, H] and their bytes
    [E, H/32, 2I], [E, I/32, H] -> y [T, H] FP64."""
    idx, p = route(x @ router.T, k, renormalize)
    y = np.zeros_like(x)
    inner = w2.shape[1]
    for e in range(w13.shape[0]):
        t, slot = np.nonzero(idx == e)
        if not len(t):
            continue
        gu = x[t] @ values(w13[e], e13[e], 0)
        g, u = gu[:, :inner], gu[:, inner:]
        h = g / (1.0 + np.exp(-g)) * u
        y[t] += p[t, slot][:, None] * (h @ values(w2[e], e2[e], 0))
    return y
