"""What the binding refuses of the int8 operators and the block norm before a raw
pointer reaches the library, with stand-in tensors (no device needed)."""
import pytest

import weight_only_int4_gb300 as w4

torch = pytest.importorskip("torch")
from test_binding_checks import Tensor, lib, operands  # noqa: E402,F401

bf16, f16, f32, i8, u8 = torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.uint8

NORM = dict(residual=((3, 64), f32), weight=((64,), bf16), h=((3, 64), bf16), after=((64,), bf16),
            gate=((3, 1), bf16))
CALLS = {
    "int8_quantize": (lambda o, **kw: w4.int8_quantize(o["x"], **kw), dict(x=((5, 128), bf16)),
                      [((5, 128), i8), ((5,), f32)], False),
    "int8_dequant": (lambda o, **kw: w4.int8_dequant(o["codes"], o["scale"], **kw),
                     dict(codes=((5, 128), i8), scale=((5,), f32)), [((5, 128), bf16)], False),
    "int8_matmul": (lambda o, **kw: w4.int8_matmul(o["a"], o["sa"], o["b"], o["sb"], **kw),
                    dict(a=((5, 128), i8), sa=((5,), f32), b=((64, 128), i8), sb=((64,), f32)), [((5, 64), bf16)], True),
    "block_norm": (lambda o, **kw: w4.block_norm(**o, **kw), NORM, [((3, 64), f32), ((3, 64), bf16)], False),
    "block_norm, codes": (lambda o, **kw: w4.block_norm(**o, quantize=True, **kw), NORM,
                          [((3, 64), f32), ((3, 64), i8), ((3,), f32)], False),
    "block_norm, residual": (lambda o, **kw: w4.block_norm(**o, **kw), {k: v for k, v in NORM.items() if k != "weight"},
                             [((3, 64), f32)], False),
}


def outputs(specs):
    made = tuple(Tensor(s, d) for s, d in specs)
    return made[0] if len(made) == 1 else made


@pytest.mark.parametrize("name", list(CALLS))
def test_operands(name, lib):  # noqa: F811
    call, spec, outs, takes_workspace = CALLS[name]
    kw = dict(workspace=Tensor((1 << 20,), u8)) if takes_workspace else {}
    call(operands(spec), out=outputs(outs), **kw)
    assert len(lib.launched) == 1
    for bad in spec:
        for how in (dict(where=-1), dict(where=1), dict(contiguous=False)):
            with pytest.raises(ValueError):
                call(operands(spec, bad, **how), out=outputs(outs), **kw)
        s, d = spec[bad]
        for other in (Tensor((*s, 1), d), Tensor((*s[:-1], s[-1] + 1), d), Tensor(s, torch.float64)):
            if bad == "x" and other.dtype == d and len(other.shape) == 2 or len(spec) == 1 and other.dtype == d:
                continue   # another shape is another call
            with pytest.raises((ValueError, TypeError)):
                call(dict(operands(spec), **{bad: other}), out=outputs(outs), **kw)
    assert len(lib.launched) == 1


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs(name, lib):  # noqa: F811
    call, spec, outs, takes_workspace = CALLS[name]
    kw = dict(workspace=Tensor((1 << 20,), u8)) if takes_workspace else {}
    for i, (s, d) in enumerate(outs):
        for bad in (Tensor(s, d, -1), Tensor(s, d, 1), Tensor(s, d, 0, False), Tensor((*s[:-1], s[-1] - 1), d),
                    Tensor(s, torch.float64)):
            made = [Tensor(*o) for o in outs]
            made[i] = bad
            with pytest.raises((ValueError, TypeError)):
                call(operands(spec), out=made[0] if len(made) == 1 else tuple(made), **kw)
    if len(outs) > 1:
        with pytest.raises(ValueError):
            call(operands(spec), out=tuple(Tensor(*o) for o in outs[:-1]), **kw)
    assert not lib.launched


def test_workspace(lib):  # noqa: F811
    call, spec, outs, _ = CALLS["int8_matmul"]
    for ws in (Tensor((1 << 20,), u8, -1), Tensor((1 << 20,), u8, 1), Tensor((1 << 20,), u8, 0, False)):
        with pytest.raises(ValueError):
            call(operands(spec), out=outputs(outs), workspace=ws)
    assert not lib.launched


def test_norm_arguments_that_do_not_go_together(lib):  # noqa: F811
    o = operands(NORM)
    for kw in (dict(residual=o["residual"]), dict(residual=o["residual"], weight=o["weight"], after=o["after"]),
               dict(residual=o["residual"], weight=o["weight"], gate=o["gate"]),
               dict(residual=o["residual"], h=o["h"], quantize=True),
               dict(residual=o["residual"], weight=o["weight"], out=(Tensor((3, 64), f32), Tensor((3, 64), bf16)))):
        with pytest.raises(ValueError):
            w4.block_norm(**kw)
    with pytest.raises(TypeError):   # a 16-bit residual beside FP32 activations
        w4.block_norm(Tensor((3, 64), bf16), Tensor((64,), f32))
    assert not lib.launched
    r = Tensor((3, 64), bf16)
    assert w4.block_norm(r, Tensor((64,), bf16), out=(None, Tensor((3, 64), bf16)))[0] is r


def test_refused_by_the_library():
    """The same errors as every other entry point: the status's name."""
    for name in ("int8_quantize", "int8_dequant", "int8_matmul", "block_norm"):
        assert f"w4a16_{name}" in w4.SIGNATURES
        assert w4.W4A16Error(f"w4a16_{name}", w4.ERR_SHAPE).status == w4.ERR_SHAPE
