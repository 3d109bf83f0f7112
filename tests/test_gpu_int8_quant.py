"""int8 rows on the device, bit for bit against the oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from oracle import int8_oracle as I8  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def guarded(shape, dtype, fill):
    """A view in the middle of a larger buffer, 16-byte aligned."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), fill, dtype=dtype, device="cuda")
    return buf, buf[64:64 + n].view(shape)


def untouched(buf, fill):
    return bool((buf[:64] == fill).all()) and bool((buf[-64:] == fill).all())


def check(x):
    """x on the CPU; codes and scales equal the oracle's."""
    want_c, want_s = I8.quantize_rows(x.double().numpy())
    cb, codes = guarded(x.shape, torch.int8, 77)
    sb, scale = guarded((x.shape[0],), torch.float32, -5.0)
    w4.int8_quantize(x.cuda(), out=(codes, scale))
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scale.cpu().numpy(), want_s, equal_nan=True)
    assert untouched(cb, 77) and untouched(sb, -5.0)
    return codes, scale


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 32), (1, 5376), (77, 2608), (33, 8192), (5, 8208), (4, 16400),
                                       (3, 32768), (2, 32784), (2, 131056), (600, 48)])
def test_shapes(dtype, rows, cols):
    gen = torch.Generator().manual_seed(rows * cols)
    x = torch.randn((rows, cols), generator=gen) * torch.exp(4 * torch.randn((rows, 1), generator=gen))
    check(x.to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_and_neighbours(dtype):
    """Rows whose largest value makes many quotients whole or half, and the values next to them."""
    info = torch.finfo(dtype)
    tops = [1.0, 127.0, 254.0, 63.5, 1.984375, 2.0, 3.0, 0.9921875, 2.0 ** -10, 100.0]
    rows = []
    for top in tops:
        k = torch.arange(0, 128, dtype=torch.float64)
        half = ((k + 0.5) / 127 * top)
        near = torch.cat([half, half * (1 + info.eps), half * (1 - info.eps), half * (1 + 3 * info.eps), k / 127 * top])
        near = near.clamp(max=top)
        row = torch.cat([torch.tensor([top], dtype=torch.float64), near, -near])
        rows.append(torch.cat([row, torch.zeros(-len(row) % 16, dtype=torch.float64)]))
    check(torch.stack(rows).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_rows(dtype):
    """Zeros, the smallest and the largest values, infinities and NaN, each beside ordinary rows."""
    info = torch.finfo(dtype)
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((12, 528), generator=gen).to(dtype)
    x[1] = 0
    x[2] = x[2].sign() * info.max
    x[3] = (x[3].double() * 2.0 ** (-20 if dtype == torch.float16 else -130)).to(dtype)
    x[4] = 0
    x[4, 100] = info.smallest_normal * info.eps      # the smallest subnormal
    x[5, 527] = float("inf")
    x[6, 0] = float("-inf")
    x[7, 263] = float("nan")
    x[8, :] = float("nan")
    x[9] = -x[9].abs()
    x[10, 5] = info.max
    check(x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 16), (77, 2608), (9, 16400)])
def test_dequant(dtype, rows, cols):
    gen = torch.Generator().manual_seed(3)
    codes = torch.randint(-128, 128, (rows, cols), generator=gen, dtype=torch.int8)
    scale = torch.rand(rows, generator=gen) * 1e-2
    yb, y = guarded((rows, cols), dtype, -5.0)
    w4.int8_dequant(codes.cuda(), scale.cuda(), out=y)
    want = (codes.float() * scale[:, None]).to(dtype)      # one FP32 product, rounded
    assert torch.equal(y.cpu(), want) and untouched(yb, -5.0)
    scale[0] = float("nan")
    assert bool(w4.int8_dequant(codes.cuda(), scale.cuda(), out_dtype=dtype)[0].isnan().all())


def test_quantised_values_of_codes_are_kept():
    """Codes times a power of two, with 127 among them, come back as they were."""
    gen = torch.Generator().manual_seed(4)
    codes = torch.randint(-127, 128, (9, 256), generator=gen, dtype=torch.int8)
    codes[:, 3] = 127
    got, scale = w4.int8_quantize((codes.float() * 0.25).cuda())
    assert torch.equal(got.cpu(), codes) and bool((scale == 0.25).all())


def test_past_32_bits():
    """More than 2^32 elements: the last rows are as right as the first."""
    rows, cols = 65600, 65536
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[:8].normal_()
    x[8:-8].fill_(1.0)
    x[-8:].normal_()
    codes, scale = w4.int8_quantize(x)
    for part in (slice(0, 8), slice(rows - 8, rows)):
        c, s = I8.quantize_rows(x[part].double().cpu().numpy())
        assert np.array_equal(codes[part].cpu().numpy(), c) and np.array_equal(scale[part].cpu().numpy(), s)
    assert bool((codes[8:-8:97] == 127).all())
    y = w4.int8_dequant(codes, scale, out=x)
    assert torch.equal(y[-8:], (codes[-8:].float() * scale[-8:, None]).bfloat16())
