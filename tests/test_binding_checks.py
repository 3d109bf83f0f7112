"""What the binding refuses before a raw pointer reaches the library: tensors and
workspaces that are not on the current CUDA device, outputs of another shape or
type. Tensors are stand-ins, so no device is needed; the library is one that
fails the test when an entry point that launches is called."""
import types

import pytest

import weight_only_int4_gb300 as w4

torch = pytest.importorskip("torch")


class Tensor:
    def __init__(self, shape, dtype, where=0, contiguous=True):
        self.shape, self.dtype, self.where, self.contiguous = torch.Size(shape), dtype, where, contiguous
        self.device = types.SimpleNamespace(index=where, type="cuda" if where >= 0 else "cpu")
        self.is_cuda = where >= 0

    def get_device(self):
        return self.where

    def is_contiguous(self):
        return self.contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 0x10000


class Library:
    """Reaching an entry point is what every test here rules out, or looks for."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("workspace_bytes"):
                return 4096
            self.launched.append(name)
            return w4.OK
        return entry


@pytest.fixture
def lib(monkeypatch):
    w4._torch()
    made = Library()
    monkeypatch.setattr(w4, "load_library", lambda: made)
    monkeypatch.setattr(w4, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(w4, "_stream_ptr", lambda stream=None: 0)
    return made


bf16, f16, i32, u8 = torch.bfloat16, torch.float16, torch.int32, torch.uint8

# operands by name, output's name, shape and type
CALLS = {
    "gemv": (lambda o, **kw: w4.gemv(o["x"], o["qweight"], o["scales"], o["qzeros"], 32, **kw),
             dict(x=((2, 128), f16), qweight=((16, 64), i32), scales=((4, 64), f16), qzeros=((4, 8), i32)),
             ((2, 64), f16), True),
    "gemm": (lambda o, **kw: w4.gemm(o["x"], o["qweight"], o["scales"], None, 32, **kw),
             dict(x=((20, 128), bf16), qweight=((16, 64), i32), scales=((4, 64), bf16)), ((20, 64), bf16), True),
    "dequant": (lambda o, **kw: w4.dequant(o["qweight"], o["scales"], None, 32, **kw),
                dict(qweight=((16, 64), i32), scales=((4, 64), bf16)), ((128, 64), bf16), False),
    "pack": (lambda o, **kw: w4.pack(o["codes"], 0, **kw), dict(codes=((64, 32), u8)), ((8, 32), i32), False),
    "unpack": (lambda o, **kw: w4.unpack(o["words"], 1, **kw), dict(words=((64, 4), i32)), ((64, 32), u8), False),
    "mxfp4_gemv": (lambda o, **kw: w4.mxfp4_gemv(o["x"], o["qweight"], o["escale"], **kw),
                   dict(x=((2, 128), bf16), qweight=((16, 64), i32), escale=((4, 64), u8)), ((2, 64), bf16), True),
    "mxfp4_gemm": (lambda o, **kw: w4.mxfp4_gemm(o["x"], o["qweight"], o["escale"], **kw),
                   dict(x=((20, 128), bf16), qweight=((16, 64), i32), escale=((4, 64), u8)), ((20, 64), bf16), True),
    "mxfp4_dequant": (lambda o, **kw: w4.mxfp4_dequant(o["qweight"], o["escale"], **kw),
                      dict(qweight=((16, 64), i32), escale=((4, 64), u8)), ((128, 64), bf16), False),
    "mxfp4_dequant_rows": (lambda o, **kw: w4.mxfp4_dequant_rows(o["codes"], o["scales"], **kw),
                           dict(codes=((5, 16), i32), scales=((1, 1, 32, 4, 4), u8)), ((5, 128), bf16), False),
    "mxfp4_tile_scales": (lambda o, **kw: w4.mxfp4_tile_scales(o["escale"], **kw), dict(escale=((5, 4), u8)),
                          ((1, 1, 32, 4, 4), u8), False),
    "mxfp4_matmul": (lambda o, **kw: w4.mxfp4_matmul(o["a"], o["ea"], o["b"], o["eb"], **kw),
                     dict(a=((5, 16), i32), ea=((1, 1, 32, 4, 4), u8), b=((64, 16), i32), eb=((1, 1, 32, 4, 4), u8)),
                     ((5, 64), bf16), True),
    "mxfp4_matmul, 40 rows": (lambda o, **kw: w4.mxfp4_matmul(o["a"], o["ea"], o["b"], o["eb"], **kw),
                              dict(a=((40, 16), i32), ea=((1, 1, 32, 4, 4), u8), b=((64, 16), i32),
                                   eb=((1, 1, 32, 4, 4), u8)), ((40, 64), bf16), True),
    "mxfp4_moe": (lambda o, **kw: w4.mxfp4_moe(o["x"], o["router"], o["w13"], o["e13"], o["w2"], o["e2"], 2, **kw),
                  dict(x=((3, 64), bf16), router=((4, 64), bf16), w13=((4, 8, 64), i32), e13=((4, 2, 64), u8),
                       w2=((4, 4, 64), i32), e2=((4, 1, 64), u8)), ((3, 64), bf16), True),
}


def operands(spec, bad=None, **how):
    return {n: Tensor(s, d, **(how if n == bad else {})) for n, (s, d) in spec.items()}


@pytest.mark.parametrize("name", list(CALLS))
def test_operands(name, lib):
    call, spec, (shape, dtype), takes_workspace = CALLS[name]
    kw = dict(workspace=Tensor((1 << 20,), u8)) if takes_workspace else {}
    out = Tensor(shape, dtype)
    call(operands(spec), out=out, **kw)
    assert len(lib.launched) == 1          # the stand-ins are accepted as they are ...
    for bad in spec:                       # ... and refused elsewhere or not dense
        for how in (dict(where=-1), dict(where=1), dict(contiguous=False)):
            with pytest.raises(ValueError):
                call(operands(spec, bad, **how), out=out, **kw)
    assert len(lib.launched) == 1


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs(name, lib):
    call, spec, (shape, dtype), takes_workspace = CALLS[name]
    kw = dict(workspace=Tensor((1 << 20,), u8)) if takes_workspace else {}
    other = torch.float64
    short = (*shape[:-1], shape[-1] - 1)
    for out in (Tensor(shape, dtype, -1), Tensor(shape, dtype, 1), Tensor(shape, dtype, 0, False), Tensor(short, dtype),
                Tensor(shape, other)):
        with pytest.raises((ValueError, TypeError)):
            call(operands(spec), out=out, **kw)
    assert not lib.launched


@pytest.mark.parametrize("name", [n for n in CALLS if CALLS[n][3]])
def test_workspaces(name, lib):
    call, spec, (shape, dtype), _ = CALLS[name]
    for ws in (Tensor((1 << 20,), u8, -1), Tensor((1 << 20,), u8, 1), Tensor((1 << 20,), u8, 0, False)):
        with pytest.raises(ValueError):
            call(operands(spec), out=Tensor(shape, dtype), workspace=ws)
    assert not lib.launched


def test_quantised_outputs(lib):
    x = Tensor((5, 128), bf16)
    good = Tensor((5, 16), i32), Tensor((1, 1, 32, 4, 4), u8)
    w4.mxfp4_quantize(x, 1, out=good)
    assert lib.launched == ["w4a16_mxfp4_quantize"]
    for i in (0, 1):
        for where in (-1, 1):
            out = list(good)
            out[i] = Tensor(out[i].shape, out[i].dtype, where)
            with pytest.raises(ValueError):
                w4.mxfp4_quantize(x, 1, out=tuple(out))
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(Tensor((5, 128), bf16, 1), 1, out=good)
    assert len(lib.launched) == 1


@pytest.mark.parametrize("name", list(CALLS))
def test_host_tensors_without_a_device(name):
    """The same answer on a host that has no CUDA driver to ask."""
    call, spec, _, _ = CALLS[name]
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        call({n: torch.zeros(s, dtype=d) for n, (s, d) in spec.items()})
