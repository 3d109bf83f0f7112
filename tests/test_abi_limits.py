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
