"""Sizes at the top of the accepted range, on the host: a dimension that a kernel
would round up past 2^31 - 1 is refused. Every call below has a misaligned
output, so that one that got past the shape check would end there, with
another status, and launch nothing."""
import os

import pytest

import weight_only_int4_gb300 as w4
from weight_only_int4_gb300 import build as w4build

P, MIS = 0x10000, 0x10008
TOP = 1 << 31
LIMIT = TOP - 512


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        w4build.build()
    return w4.load_library()


def product(lib, M=5, N=64, K=128):
    return lib.w4a16_mxfp4_matmul(P, P, P, P, MIS, M, N, K, w4.BF16, P, 1 << 40, None)


def test_mxfp4_product(lib):
    for M in (TOP - 1, TOP - 128, TOP - 255, TOP - 256, LIMIT + 1):
        assert product(lib, M=M, K=32) == w4.ERR_SHAPE, M
    for N in (TOP - 8, TOP - 128, TOP - 256, LIMIT + 8):
        assert product(lib, N=N, K=32) == w4.ERR_SHAPE, N
    for K in (TOP - 32, TOP - 256, LIMIT + 32):
        assert product(lib, K=K) == w4.ERR_SHAPE, K
    assert product(lib, M=LIMIT, K=32) == product(lib, N=LIMIT, K=32) == product(lib, K=LIMIT) == w4.ERR_ALIGN


def layer(lib, fn, M=5, N=64, K=128):
    if fn.startswith("w4a16_mxfp4"):
        return getattr(lib, fn)(P, P, P, MIS, M, N, K, P, 1 << 40, None)
    return getattr(lib, fn)(P, P, P, P, MIS, M, N, K, 32, w4.BF16, P, 1 << 40, None)


@pytest.mark.parametrize("fn", ["w4a16_gemv", "w4a16_gemm", "w4a16_mxfp4_gemv", "w4a16_mxfp4_gemm"])
def test_layers(lib, fn):
    if fn.endswith("gemm"):
        for M in (TOP - 1, TOP - 255, TOP - 256, LIMIT + 1):
            assert layer(lib, fn, M=M, K=32) == w4.ERR_SHAPE, M
        assert layer(lib, fn, M=LIMIT, K=32) == w4.ERR_ALIGN
    for N in (TOP - 16, TOP - 128, TOP - 256, LIMIT + 16):
        assert layer(lib, fn, N=N, K=32) == w4.ERR_SHAPE, N
    for K in (TOP - 32, TOP - 256, LIMIT + 32):
        assert layer(lib, fn, K=K) == w4.ERR_SHAPE, K
    assert layer(lib, fn, N=LIMIT, K=32) == layer(lib, fn, K=LIMIT) == w4.ERR_ALIGN
