"""CPU checks of the MXFP4 operators' entry points: every bad argument is
refused on the host, before the device gate."""
import os

import pytest

import weight_only_int4_gb300 as w4
from weight_only_int4_gb300 import build as w4build

# Pointers that are never dereferenced: every call below ends at a host check.
P = 0x10000
MIS = 0x10008


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        w4build.build()
    return w4.load_library()


def quantize(lib, **kw):
    a = dict(x=P, c=P, e=P, rows=64, cols=64, dim=1, dt=w4.BF16)
    a.update(kw)
    return lib.w4a16_mxfp4_quantize(a["x"], a["c"], a["e"], a["rows"], a["cols"], a["dim"], a["dt"], None)


@pytest.mark.parametrize("dim", [0, 1])
def test_quantize_rejections(lib, dim):
    for name in ("x", "c", "e"):
        assert quantize(lib, dim=dim, **{name: None}) == w4.ERR_NULL
        assert quantize(lib, dim=dim, **{name: MIS}) == w4.ERR_ALIGN
    assert quantize(lib, dim=dim, dt=3) == w4.ERR_DTYPE
    assert quantize(lib, dim=dim, rows=0) == w4.ERR_SHAPE
    assert quantize(lib, dim=dim, cols=-32) == w4.ERR_SHAPE
    assert quantize(lib, dim=dim, rows=1 << 31) == w4.ERR_SHAPE
    assert quantize(lib, dim=2) == w4.ERR_SHAPE
    if dim == 0:
        assert quantize(lib, dim=0, rows=48) == w4.ERR_SHAPE      # whole blocks of 32 rows
        assert quantize(lib, dim=0, cols=24) == w4.ERR_SHAPE      # exponent rows start 16-byte aligned
    else:
        assert quantize(lib, dim=1, cols=48) == w4.ERR_SHAPE      # whole blocks of 32 columns


def test_row_layout_rejections(lib):
    d = lambda **k: lib.w4a16_mxfp4_dequant_rows(k.get("c", P), k.get("e", P), k.get("w", P), k.get("rows", 5),
                                                 k.get("cols", 64), None)
    t = lambda **k: lib.w4a16_mxfp4_tile_scales(k.get("src", P), k.get("dst", P), k.get("rows", 5),
                                                k.get("cols", 64), None)
    for name in ("c", "e", "w"):
        assert d(**{name: None}) == w4.ERR_NULL
        assert d(**{name: MIS}) == w4.ERR_ALIGN
    assert t(src=None) == w4.ERR_NULL and t(dst=None) == w4.ERR_NULL
    assert t(dst=MIS) == w4.ERR_ALIGN
    for f in (d, t):
        assert f(rows=0) == w4.ERR_SHAPE
        assert f(cols=40) == w4.ERR_SHAPE


def matmul(lib, **kw):
    a = dict(a=P, ea=P, b=P, eb=P, y=P, M=5, N=64, K=128, dt=w4.BF16, ws=P, n=1 << 40)
    a.update(kw)
    return lib.w4a16_mxfp4_matmul(a["a"], a["ea"], a["b"], a["eb"], a["y"], a["M"], a["N"], a["K"], a["dt"], a["ws"],
                                  a["n"], None)


def test_matmul_rejections(lib):
    for name in ("a", "ea", "b", "eb", "y"):
        assert matmul(lib, **{name: None}) == w4.ERR_NULL
        assert matmul(lib, **{name: MIS}) == w4.ERR_ALIGN
    assert matmul(lib, dt=3) == w4.ERR_DTYPE
    assert matmul(lib, M=0) == w4.ERR_SHAPE
    assert matmul(lib, N=12) == w4.ERR_SHAPE
    assert matmul(lib, K=48) == w4.ERR_SHAPE
    assert matmul(lib, K=-32) == w4.ERR_SHAPE
    assert matmul(lib, N=1 << 31) == w4.ERR_SHAPE
    # exponent tiles past 32-bit coordinates
    assert matmul(lib, N=(1 << 31) - 8, K=(1 << 31) - 32) == w4.ERR_SHAPE
    assert matmul(lib, ws=None) == w4.ERR_WORKSPACE      # M <= 128 always needs one
    assert matmul(lib, ws=MIS) == w4.ERR_WORKSPACE


def moe(lib, **kw):
    a = dict(x=P, r=P, w13=P, e13=P, w2=P, e2=P, y=P, T=3, E=8, k=2, H=64, I=32, ws=P, n=1 << 40)
    a.update(kw)
    return lib.w4a16_mxfp4_moe(a["x"], a["r"], a["w13"], a["e13"], a["w2"], a["e2"], a["y"], a["T"], a["E"], a["k"],
                               a["H"], a["I"], 1, a["ws"], a["n"], None)


def test_moe_rejections(lib):
    for name in ("x", "r", "w13", "e13", "w2", "e2", "y"):
        assert moe(lib, **{name: None}) == w4.ERR_NULL
        assert moe(lib, **{name: MIS}) == w4.ERR_ALIGN
    for bad in (dict(T=0), dict(T=65), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(k=17, E=32), dict(H=48),
                dict(H=0), dict(H=65568), dict(I=40), dict(I=-32), dict(I=1 << 31)):
        assert moe(lib, **bad) == w4.ERR_SHAPE, bad
        shape = dict(T=3, E=8, k=2, H=64, I=32, **{}) | bad
        assert lib.w4a16_mxfp4_moe_workspace_bytes(shape["T"], shape["E"], shape["k"], shape["H"], shape["I"]) == 0
    assert moe(lib, ws=None) == w4.ERR_WORKSPACE
    assert moe(lib, ws=MIS) == w4.ERR_WORKSPACE
    need = lib.w4a16_mxfp4_moe_workspace_bytes(3, 8, 2, 64, 32)
    assert need > 0
    assert moe(lib, n=need - 1) == w4.ERR_WORKSPACE
