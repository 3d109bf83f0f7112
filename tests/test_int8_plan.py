"""Which way the int8 product runs a shape, on the host: the shapes of the GPU tests reach
every way that any shape reaches, and what the kernels rely on holds on any device."""
import ctypes
import os
import random

import pytest

import weight_only_int4_gb300 as w4
from weight_only_int4_gb300 import build as w4build

SMS = 152

# (M, N, K): (rows per tile, split, shared, rows per tile of the pairs, columns on them)
PLANS = {
    (1, 520, 1040): (-1, 1, 0, 0, 0),
    (2, 520, 1040): (-1, 1, 0, 0, 0),
    (3, 520, 1040): (-1, 1, 0, 0, 0),
    (4, 520, 1040): (-1, 1, 0, 0, 0),
    (5, 520, 1040): (-1, 1, 0, 0, 0),
    (7, 40, 8208): (-1, 1, 0, 0, 0),
    (13, 264, 8208): (-1, 1, 0, 0, 0),
    # 128 rows of B per tile: one tile a CTA, several, a cluster per tile, shared units
    (9, 10960, 272): (16, 1, 0, 0, 0),
    (20, 31576, 528): (32, 1, 0, 0, 0),
    (11, 31312, 1296): (16, 1, 0, 0, 0),
    (51, 31232, 672): (64, 1, 0, 0, 0),
    (92, 36872, 1552): (128, 1, 0, 0, 0),
    (9, 1640, 5120): (16, 8, 0, 0, 0),
    (12, 6400, 5376): (16, 3, 0, 0, 0),
    (17, 8, 960): (32, 4, 0, 0, 0),
    (64, 4104, 4112): (64, 4, 0, 0, 0),
    (71, 3232, 6160): (128, 5, 0, 0, 0),
    (315, 2560, 12208): (128, 2, 0, 0, 0),
    (16, 20488, 1040): (16, 1, 1, 0, 0),
    (30, 43008, 272): (32, 1, 1, 0, 0),
    (64, 20488, 656): (64, 1, 1, 0, 0),
    (128, 20488, 656): (128, 1, 1, 0, 0),
    (40, 264, 272): (32, 1, 0, 0, 0),
    (4867, 40, 272): (64, 1, 0, 0, 0),
    # pairs: every height, one wave and several, all columns and whole waves of them
    (65, 10016, 272): (0, 1, 0, 96, 10016),
    (262, 10360, 144): (0, 1, 0, 96, 10360),
    (5077, 136, 272): (0, 1, 0, 128, 136),
    (290, 9848, 272): (0, 1, 0, 128, 9848),
    (4978, 264, 144): (0, 1, 0, 160, 264),
    (129, 21240, 400): (0, 1, 0, 160, 21240),
    (161, 9960, 272): (0, 1, 0, 192, 9960),
    (171, 20128, 272): (0, 1, 0, 192, 20128),
    (196, 9760, 272): (0, 1, 0, 224, 9760),
    (194, 21560, 144): (0, 1, 0, 224, 21560),
    (243, 10160, 272): (0, 1, 0, 256, 10160),
    (229, 29232, 272): (0, 1, 0, 256, 29232),
    (241, 10112, 10944): (0, 8, 0, 128, 9728),
    (323, 13472, 11120): (0, 8, 0, 128, 12800),
    (138, 19992, 2464): (0, 8, 0, 160, 19456),
    (258, 20152, 2672): (0, 8, 0, 160, 19456),
    (174, 21496, 2256): (0, 4, 0, 192, 19456),
    (341, 20400, 2256): (0, 6, 0, 192, 19456),
    (201, 20000, 2368): (0, 8, 0, 224, 19456),
    (205, 40144, 1952): (0, 7, 0, 224, 38912),
    (255, 21192, 2336): (0, 5, 0, 256, 19456),
    (469, 20376, 1936): (0, 4, 0, 256, 19456),
    (226, 24656, 13664): (0, 1, 0, 256, 19456),
    (497, 23432, 11536): (0, 1, 0, 256, 19456),
    # 32 chunks of rows, one row in the last
    (253953, 264, 16): (0, 1, 0, 224, 264),
}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        w4build.build()
    return w4.load_library()


def plan(lib, M, N, K, sms=SMS):
    out = (ctypes.c_int * 5)()
    assert lib.w4a16_selftest_int8_matmul_plan(M, N, K, sms, out) == w4.OK
    return tuple(out)


def kind(M, N, K, p, sms=SMS):
    mp, split, shared, bm, columns = p
    if mp < 0:
        return "dots", M if M <= 4 else 6 if M <= 6 else 8 if M <= 8 else 16
    if mp:
        tiles = -(-M // mp) * -(-N // 128)
        return "tiles", mp, "cluster" if split > 1 else "shared" if shared else "several" if tiles > sms else "one"
    tiles = -(-min(M, 8192) // bm) * -(-columns // 256)
    return "pairs", bm, (split > 1, "cut") if columns < N else "whole", "one" if tiles <= sms // 2 else "several"


def draws(seed, count, top=(13, 15.4, 14.4)):
    rng = random.Random(seed)
    for _ in range(count):
        M, N, K = (int(2 ** rng.uniform(0, t)) for t in top)
        yield M, max(8, N // 8 * 8), max(16, K // 16 * 16)


@pytest.mark.parametrize("shape", list(PLANS))
def test_shapes_of_the_gpu_tests(lib, shape):
    assert plan(lib, *shape) == PLANS[shape]


def test_every_way_is_among_them(lib):
    seen = {kind(*s, plan(lib, *s)) for s in draws(1, 150000)}
    assert seen <= {kind(*s, p) for s, p in PLANS.items()}


@pytest.mark.parametrize("sms", [1, 2, 20, 76, 132, 148, 152, 160])
def test_what_the_kernels_rely_on(lib, sms):
    for M, N, K in draws(sms, 20000, (18, 18, 17)):
        K = min(K, 131056)
        mp, split, shared, bm, columns = plan(lib, M, N, K, sms)
        assert mp in (-1, 0, 16, 32, 64, 128) and 1 <= split <= 8 and not (split > 1 and shared)
        assert mp >= 0 or M <= 16
        assert (mp == 0) == (bm > 0)
        if mp == 0:   # a tile's rows halve into whole groups of 16; columns go in whole tiles, some to the pairs at least
            assert bm % 32 == 0 and 32 <= bm <= 256
            assert 0 < columns <= N and (columns == N or columns % 256 == 0)
        if shared:
            assert M <= mp and -(-N // 128) > sms


def test_refusals(lib):
    out = (ctypes.c_int * 5)()
    assert lib.w4a16_selftest_int8_matmul_plan(1, 8, 16, SMS, None) == w4.ERR_NULL
    for bad in ((0, 8, 16, SMS), (1, 12, 16, SMS), (1, 8, 24, SMS), (1, 8, 131072, SMS), (1, 8, 16, 0)):
        assert lib.w4a16_selftest_int8_matmul_plan(*bad, out) == w4.ERR_SHAPE


@pytest.mark.parametrize("sms", [20, 148, 152, 160])
def test_up_to_four_rows_need_no_workspace(lib, sms):
    """The binding does not ask for their workspace."""
    for _, N, K in draws(sms, 2000, (1, 18, 17)):
        for M in (1, 2, 3, 4):
            assert plan(lib, M, N, min(K, 131056), sms) == (-1, 1, 0, 0, 0)
