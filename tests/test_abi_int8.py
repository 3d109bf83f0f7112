"""CPU checks of the int8 operators' entry points and of the block norm's: every
bad argument is refused on the host, before the device gate."""
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


@pytest.mark.parametrize("name", ["w4a16_int8_quantize", "w4a16_int8_dequant"])
def test_row_rejections(lib, name):
    def call(p0=P, p1=P, p2=P, rows=5, cols=64, dt=w4.BF16):
        return getattr(lib, name)(p0, p1, p2, rows, cols, dt, None)
    for i in range(3):
        assert call(**{f"p{i}": None}) == w4.ERR_NULL
        assert call(**{f"p{i}": MIS}) == w4.ERR_ALIGN
    assert call(dt=3) == w4.ERR_DTYPE
    for bad in (dict(rows=0), dict(rows=-1), dict(cols=0), dict(cols=24), dict(cols=-16), dict(rows=1 << 31),
                dict(cols=1 << 31)):
        assert call(**bad) == w4.ERR_SHAPE, bad


def matmul(lib, **kw):
    a = dict(a=P, sa=P, b=P, sb=P, y=P, M=5, N=64, K=128, dt=w4.BF16, ws=P, n=1 << 40)
    a.update(kw)
    return lib.w4a16_int8_matmul(a["a"], a["sa"], a["b"], a["sb"], a["y"], a["M"], a["N"], a["K"], a["dt"], a["ws"],
                                 a["n"], None)


def test_matmul_rejections(lib):
    for name in ("a", "sa", "b", "sb", "y"):
        assert matmul(lib, **{name: None}) == w4.ERR_NULL
        assert matmul(lib, **{name: MIS}) == w4.ERR_ALIGN
    assert matmul(lib, ws=MIS) == w4.ERR_ALIGN
    assert matmul(lib, dt=3) == w4.ERR_DTYPE
    for bad in (dict(M=0), dict(N=12), dict(N=-8), dict(K=24), dict(K=0), dict(K=131072), dict(M=1 << 31),
                dict(N=1 << 31), dict(M=(1 << 31) - 8)):
        assert matmul(lib, **bad) == w4.ERR_SHAPE, bad
        shape = dict(M=5, N=64, K=128) | bad
        assert lib.w4a16_int8_matmul_workspace_bytes(shape["M"], shape["N"], shape["K"]) == 0


def norm(lib, **kw):
    a = dict(r=P, rdt=w4.BF16, h=P, after=P, gate=P, kind=w4.GATE_CHANNEL, scale=1.0, ro=P, w=P, eps=1e-6, y=P, c=None,
             cs=None, T=3, H=64, dt=w4.BF16)
    a.update(kw)
    return lib.w4a16_block_norm(a["r"], a["rdt"], a["h"], a["after"], a["gate"], a["kind"], a["scale"], a["ro"], a["w"],
                                a["eps"], a["y"], a["c"], a["cs"], a["T"], a["H"], a["dt"], None)


def test_norm_rejections(lib):
    codes = dict(y=None, c=P, cs=P)
    bare = dict(h=None, after=None, gate=None, ro=None)
    for bad in (dict(r=None), dict(ro=None), dict(y=None), dict(codes, c=None), dict(codes, cs=None),
                dict(bare, w=None, y=None)):
        assert norm(lib, **bad) == w4.ERR_NULL, bad
    for bad in (dict(dt=3), dict(rdt=w4.F16), dict(dt=w4.F32), dict(rdt=3)):
        assert norm(lib, **bad) == w4.ERR_DTYPE, bad
    for bad in (dict(T=0), dict(T=1 << 31), dict(H=0), dict(H=24), dict(H=16400), dict(H=-16), dict(kind=3),
                dict(kind=-1), dict(h=None), dict(bare, after=P), dict(bare, gate=P), dict(bare, ro=P),
                dict(c=P, cs=P), dict(c=P), dict(cs=P), dict(w=None), dict(codes, w=None)):
        assert norm(lib, **bad) == w4.ERR_SHAPE, bad
    for bad in (dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert norm(lib, **bad) == w4.ERR_UNSUPPORTED, bad
    for name in ("r", "h", "after", "gate", "ro", "w", "y"):
        assert norm(lib, **{name: MIS}) == w4.ERR_ALIGN, name
    for name in ("c", "cs"):
        assert norm(lib, **dict(codes, **{name: MIS})) == w4.ERR_ALIGN, name
