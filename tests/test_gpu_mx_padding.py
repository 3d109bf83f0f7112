"""The exponent tiles' padding: bytes of blocks past a row's end are written as
zero, bytes of rows past the operand's end and the memory around the tiles are
left alone. Every buffer starts as 0xFF, which none of these bytes may keep, or
must keep."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from oracle import mxfp4_ops_oracle as Q  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [(1, 32), (1, 5376), (3, 96), (31, 160), (127, 128), (128, 224), (129, 352), (300, 2080), (4100, 1056)]
PAD = 512


def filled(shape):
    buf = torch.full((int(np.prod(shape)) + 2 * PAD,), 255, dtype=torch.uint8, device="cuda")
    return buf, buf[PAD:-PAD].view(shape)


def expected(e):
    """Tiles of [R, B] bytes: zero past a row's end, 255 in rows past R."""
    R, B = e.shape
    full = np.full((-(-R // 128) * 128, -(-B // 4) * 4), 255, dtype=np.uint8)
    full[:R] = 0
    full[:R, :B] = e
    return full.reshape(-1, 4, 32, full.shape[1] // 4, 4).transpose(0, 3, 2, 1, 4)


def untouched(buf):
    return bool((buf[:PAD] == 255).all()) and bool((buf[-PAD:] == 255).all())


@pytest.mark.parametrize("R,K", [s for s in SIZES if s[0] <= 300])
def test_the_expectation_is_the_oracles(R, K):
    e = np.random.default_rng(R).integers(0, 255, size=(R, K // 32)).astype(np.uint8)
    want = expected(e)
    rows = np.broadcast_to(np.arange(want.shape[0] * 128).reshape(-1, 1, 4, 32, 1).transpose(0, 1, 3, 2, 4), want.shape)
    assert np.array_equal(np.where(rows < R, want, 0), Q.tile_scales(e))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("R,K", SIZES)
def test_quantised_rows(R, K, dtype):
    x = torch.randn((R, K), generator=torch.Generator().manual_seed(R + K)).to(DTYPES[dtype])
    buf, tiles = filled(w4.mxfp4_scale_shape(R, K))
    codes = torch.empty((R, K // 8), dtype=torch.int32, device="cuda")
    w4.mxfp4_quantize(x.cuda(), 1, out=(codes, tiles))
    torch.cuda.synchronize()
    assert untouched(buf)
    assert np.array_equal(tiles.cpu().numpy(), expected(Q.quantize(x.double().numpy(), 1)[1]))


@pytest.mark.parametrize("R,K", SIZES)
def test_tiled_scales(R, K):
    e = torch.randint(0, 256, (R, K // 32), dtype=torch.uint8, generator=torch.Generator().manual_seed(R))
    buf, tiles = filled(w4.mxfp4_scale_shape(R, K))
    w4.mxfp4_tile_scales(e.cuda(), out=tiles)
    torch.cuda.synchronize()
    assert untouched(buf)
    assert np.array_equal(tiles.cpu().numpy(), expected(e.numpy()))


@pytest.mark.parametrize("M,N,K", [(3, 264, 96), (20, 136, 32), (40, 1048, 1120), (100, 12008, 1888), (700, 7696, 288)])
def test_product_over_a_last_block_of_its_own(M, N, K):
    """K % 64 == 32: the last MMA takes the padding block's bytes, whose codes are zero. Were one of them 255, its row
    or column would be NaN."""
    gen = torch.Generator().manual_seed(M)
    ops = []
    for rows in (M, N):
        x = torch.randn((rows, K), generator=gen).to(torch.bfloat16).cuda()
        _, tiles = filled(w4.mxfp4_scale_shape(rows, K))
        ops += w4.mxfp4_quantize(x, 1, out=(torch.empty((rows, K // 8), dtype=torch.int32, device="cuda"), tiles))
    y = w4.mxfp4_matmul(*ops, out_dtype=torch.float32)
    a, b = (w4.mxfp4_dequant_rows(*ops[i:i + 2]).double() for i in (0, 2))
    # K / 32 block sums, each addition within 2^-22 of the running magnitude
    bound = (K / 32 + 8) * 2.0 ** -22 * (a.abs() @ b.abs().T)
    assert bool(((y.double() - a @ b.T).abs() <= bound).all())
    assert w4.device_status() == w4.OK
