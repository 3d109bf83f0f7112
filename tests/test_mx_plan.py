"""Which way the MXFP4 product runs a shape (rows of A per tile, CTAs that split
K, shared tiles), on the host: the shapes of the GPU tests reach every way that
any shape reaches, and the ways that the kernel leaves out of a row template
are never taken."""
import ctypes
import os
import random

import pytest

import weight_only_int4_gb300 as w4
from weight_only_int4_gb300 import build as w4build

SMS = 152

# (M, N, K): (rows per tile, split, shared); `deep`: several tiles for some CTAs, more K steps than the ring holds
PLANS = {
    (128, 20480, 2080): (128, 1, 0),      # 160 tiles: two for some CTAs, nine steps
    (100, 20488, 2592): (128, 1, 0),      # the same, ragged everywhere, eleven steps
    (100, 12008, 1888): (128, 1, 0),
    (512, 4096, 4096): (128, 1, 0),
    (300, 5128, 1120): (128, 1, 0),       # three row tiles, the last of 44 rows
    (16, 20480, 5376): (16, 1, 1),        # 160 tiles of 21 steps over 152 CTAs
    (7, 43008, 1056): (16, 1, 1),         # up to four pieces of tiles a CTA
    (32, 20488, 2592): (32, 1, 1),
    (19, 21000, 4128): (32, 1, 1),
    (33, 20480, 2080): (64, 1, 0),        # two tiles for some CTAs
    (129, 2600, 2080): (64, 1, 0),
    (9, 38400, 800): (16, 1, 0),          # 300 tiles: whole ones, two a CTA
    (24, 2048, 1024): (32, 1, 0),
    (16, 2048, 5376): (16, 6, 0),
    (16, 5376, 2048): (16, 3, 0),         # six of eight steps saved
    (16, 5376, 1536): (16, 1, 0),         # four of six would be
    (50, 5376, 2048): (64, 1, 0),
    (1, 2048, 2048): (16, 4, 0),
    (17, 5376, 4128): (32, 3, 0),
    (70, 2000, 8192): (64, 4, 0),
    (700, 10240, 288): (0, 1, 0),
}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        w4build.build()
    return w4.load_library()


def plan(lib, M, N, K, sms=SMS):
    out = (ctypes.c_int * 3)()
    assert lib.w4a16_selftest_mxfp4_matmul_plan(M, N, K, sms, out) == w4.OK
    return tuple(out)


def kind(p):
    return p[0], p[1] > 1, p[2]


@pytest.mark.parametrize("shape", list(PLANS))
def test_shapes_of_the_gpu_tests(lib, shape):
    assert plan(lib, *shape) == PLANS[shape]


def test_every_way_is_among_them(lib):
    rng = random.Random(1)
    seen = set()
    for _ in range(40000):
        M, N, K = (int(2 ** rng.uniform(0, top)) for top in (12, 16.5, 15.5))
        seen.add(kind(plan(lib, M, max(8, N // 8 * 8), max(32, K // 32 * 32))))
    assert seen == {kind(p) for p in PLANS.values()}


@pytest.mark.parametrize("sms", [20, 76, 148, 152, 160])
def test_what_a_row_template_leaves_out(lib, sms):
    rng = random.Random(sms)
    for _ in range(20000):
        M, N, K = (int(2 ** rng.uniform(0, top)) for top in (13, 18, 18))
        mp, split, shared = plan(lib, M, max(8, N // 8 * 8), max(32, K // 32 * 32), sms)
        assert 1 <= split <= 6 and not (split > 1 and shared)
        assert split == 1 or mp in (16, 32, 64)
        assert not shared or (mp in (16, 32) and M <= mp)
        assert mp or M > 128


def test_refusals(lib):
    out = (ctypes.c_int * 3)()
    assert lib.w4a16_selftest_mxfp4_matmul_plan(1, 8, 32, SMS, None) == w4.ERR_NULL
    for bad in ((0, 8, 32, SMS), (1, 12, 32, SMS), (1, 8, 48, SMS), (1, 8, 32, 0)):
        assert lib.w4a16_selftest_mxfp4_matmul_plan(*bad, out) == w4.ERR_SHAPE
