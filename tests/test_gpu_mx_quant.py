"""Quantisation to MXFP4 on the GPU: codes, exponent bytes and both dense
copies equal the FP64 oracle's bit for bit, in both layouts, for each input
type, at odd sizes, at every rounding boundary and on degenerate blocks."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from gpu_util import torch_to_f64  # noqa: E402
from oracle import mxfp4_ops_oracle as Q  # noqa: E402
from oracle.mxfp4_oracle import dequantize_mx  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def make(shape, dtype, seed, spread=0.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen, dtype=torch.float64)
    if spread:
        x = x * torch.exp2(torch.randint(-int(spread), int(spread) + 1, shape, generator=gen).double())
    return x.to(DTYPES[dtype])


def check(x, dim):
    """Codes and bytes against the oracle, guards around both outputs, and the dense copy."""
    R, C = x.shape
    want_c, want_e = Q.quantize(x.double().numpy(), dim)
    want_w = Q.words(want_c, dim)
    want_s = want_e if dim == 0 else Q.tile_scales(want_e)
    pad = 64
    cbuf = torch.full((want_w.size + 2 * pad,), -77, dtype=torch.int32, device="cuda")
    ebuf = torch.full((want_s.size + 2 * pad,), 0 if dim else 99, dtype=torch.uint8, device="cuda")
    codes = cbuf[pad:-pad].view(want_w.shape)
    escale = ebuf[pad:-pad].view(want_s.shape)
    got_c, got_e = w4.mxfp4_quantize(x.cuda(), dim, out=(codes, escale))
    dense = w4.mxfp4_dequant_rows(codes, escale) if dim else w4.mxfp4_dequant(codes, escale)
    torch.cuda.synchronize()
    assert got_c.data_ptr() == codes.data_ptr() and got_e.data_ptr() == escale.data_ptr()
    for buf, v in ((cbuf, -77), (ebuf, 0 if dim else 99)):
        assert torch.all(buf[:pad] == v) and torch.all(buf[-pad:] == v), "write outside the output"
    assert np.array_equal(escale.cpu().numpy(), want_s), "exponent bytes"
    assert np.array_equal(codes.cpu().numpy().view(np.uint32), np.asarray(want_w).view(np.uint32)), "codes"
    want = Q.values(want_c, want_e, dim)
    assert np.array_equal(torch_to_f64(dense), want, equal_nan=True), "dense copy"
    if dim == 0:
        assert np.array_equal(dequantize_mx(np.asarray(want_w), want_e), want, equal_nan=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("R,K", [(1, 32), (1, 64), (3, 96), (1, 5376), (127, 128), (128, 160), (129, 224), (300, 2080)])
def test_rows(dtype, R, K):
    check(make((R, K), dtype, seed=R + K, spread=6), 1)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("K,N", [(32, 16), (64, 48), (96, 272), (160, 1040), (2080, 48)])
def test_columns(dtype, K, N):
    check(make((K, N), dtype, seed=K + N, spread=6), 0)


@pytest.mark.parametrize("dim", [0, 1])
def test_large_enough_for_every_trip_of_the_loops(dim):
    """More groups than one grid holds four times over (rows), more blocks than one grid (columns)."""
    shape = (4100, 2048) if dim else (1024, 16400)
    x = make(shape, "bf16", seed=9)
    xs = x.cuda()
    codes, escale = w4.mxfp4_quantize(xs, dim)
    dense = w4.mxfp4_dequant_rows(codes, escale) if dim else w4.mxfp4_dequant(codes, escale)
    # every value is one the oracle gives; whole rows are compared at both ends and between
    v = xs.float() if dim else xs.float().T.contiguous()
    d = dense.float() if dim else dense.float().T.contiguous()
    pick = [0, 1, v.shape[0] // 2, v.shape[0] - 2, v.shape[0] - 1]
    c, e = Q.quantize(v[pick].double().cpu().numpy(), 1)
    assert np.array_equal(d[pick].double().cpu().numpy(), Q.values(c, e, 1))
    # and every element is within the largest possible error, 2 of 4..8 steps of its block
    amax = v.reshape(v.shape[0], -1, 32).abs().amax(dim=-1, keepdim=True)
    assert bool(((d - v).reshape(v.shape[0], -1, 32).abs() <= amax / 4).all())


@pytest.mark.parametrize("dim", [0, 1])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rounding_boundaries(dim, dtype):
    """Multiples of 1/64 below 8 in blocks whose largest value is 7.75, both signs, several scales."""
    vals = torch.arange(0, 512, dtype=torch.float64) / 64.0
    vals = vals[vals <= 7.75]
    vals = torch.cat([vals, torch.zeros((-len(vals)) % 31, dtype=torch.float64)]).reshape(-1, 31)
    blocks = torch.cat([torch.full((len(vals), 1), 7.75, dtype=torch.float64), vals], dim=1)
    rows = torch.cat([blocks, -blocks, blocks * 2.0 ** -7, blocks * 2.0 ** 5])
    x = rows.to(DTYPES[dtype])
    x = x if dim else x.T.contiguous()
    if dim == 0 and x.shape[1] % 16:
        x = torch.cat([x, torch.zeros((32, 16 - x.shape[1] % 16), dtype=x.dtype)], dim=1)
    check(x.contiguous(), dim)


@pytest.mark.parametrize("dim", [0, 1])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_degenerate_blocks(dim, dtype):
    """Zeros, negative zeros, infinities, NaN, the type's extremes and subnormals, each in a block of its own."""
    t = DTYPES[dtype]
    info = torch.finfo(t)
    rows = torch.zeros((16, 32), dtype=t)
    rows[1] = -0.0
    rows[2, 5] = float("inf")
    rows[3, 31] = float("-inf")
    rows[4, 0] = float("nan")
    rows[5] = info.max
    rows[6, 3], rows[6, 4] = info.min, info.max / 2
    rows[7, 9] = info.tiny
    rows[8, 9] = info.tiny / 4                      # subnormal
    rows[9, 0], rows[9, 1] = info.max, info.tiny
    rows[10] = torch.arange(32, dtype=torch.float64).to(t) * info.tiny / 8
    rows[11, 7] = 1.0
    rows[11, 8] = float("nan")
    rows[12] = torch.linspace(-1, 1, 32, dtype=torch.float64).to(t)
    check(rows if dim else rows.T.contiguous(), dim)


def test_smallest_float_blocks():
    """FP32 blocks around the clamp of the exponent byte at 0, down to the smallest subnormal."""
    p = torch.arange(-149, -118, dtype=torch.float64)
    rows = torch.exp2(p)[:, None] * torch.linspace(0.03125, 1.0, 32, dtype=torch.float64)[None, :]
    check(rows.float(), 1)


def test_stack_of_matrices():
    x = make((3 * 64, 48), "bf16", seed=2)
    c2, e2 = w4.mxfp4_quantize(x.cuda(), 0)
    c3, e3 = w4.mxfp4_quantize(x.view(3, 64, 48).cuda(), 0)
    assert c3.shape == (3, 8, 48) and e3.shape == (3, 2, 48)
    assert torch.equal(c3.reshape(c2.shape), c2) and torch.equal(e3.reshape(e2.shape), e2)


@pytest.mark.parametrize("dim", [0, 1])
def test_quantising_a_dense_copy_gives_it_back(dim):
    x = make((256, 320), "bf16", seed=8).cuda()
    back = (lambda c, e: w4.mxfp4_dequant_rows(c, e)) if dim else (lambda c, e: w4.mxfp4_dequant(c, e))
    v = back(*w4.mxfp4_quantize(x, dim))
    assert torch.equal(back(*w4.mxfp4_quantize(v, dim)), v)


@pytest.mark.parametrize("R,K", [(1, 32), (5, 160), (128, 128), (130, 4096)])
def test_tile_scales(R, K):
    e = torch.randint(0, 256, (R, K // 32), dtype=torch.uint8, generator=torch.Generator().manual_seed(R))
    out = torch.zeros(w4.mxfp4_scale_shape(R, K), dtype=torch.uint8, device="cuda")
    got = w4.mxfp4_tile_scales(e.cuda(), out=out)
    assert np.array_equal(got.cpu().numpy(), Q.tile_scales(e.numpy()))


def test_side_stream():
    x = make((64, 4096), "bf16", seed=4).cuda()
    ref = w4.mxfp4_quantize(x, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.mxfp4_quantize(x, 1, stream=side)
    dense = w4.mxfp4_dequant_rows(*got, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0])
    assert torch.equal(dense, w4.mxfp4_dequant_rows(*ref))


def test_binding_refusals():
    x = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(x, 2)
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(x[:, :48], 1)                       # not contiguous
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(x[:40].contiguous(), 0)             # 40 rows: no whole blocks
    with pytest.raises(TypeError):
        w4.mxfp4_quantize(x.double(), 1)
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(x.cpu(), 1)
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(x[:0], 1)
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(x, 1, out=(torch.empty((64, 7), dtype=torch.int32, device="cuda"), None))
    codes, e = w4.mxfp4_quantize(x, 1)
    with pytest.raises(ValueError):
        w4.mxfp4_dequant_rows(codes, e[:, :, :, :, :2].contiguous())
    with pytest.raises(w4.W4A16Error) as err:
        w4.mxfp4_quantize(torch.zeros((32, 24), dtype=torch.bfloat16, device="cuda"), 0)   # N % 16
    assert err.value.status == w4.ERR_SHAPE
