"""Every layout of the row quantisation, bit for bit against the oracle: many rows (more
than two per SM, so that rows are held by few threads) in numbers that no block's count
of rows divides, and few."""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from test_gpu_int8_quant import check, untouched, guarded  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
# 16-bit rows: a warp holds up to 2048 elements in 1, 2, 4 or 8 vectors a thread, a block up to 65536; FP32: half of that
COLS = [16, 256, 272, 512, 528, 1024, 1040, 2048, 2064, 4096, 5376, 8208, 16384, 16400, 32768, 32784]


def values(rows, cols, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=gen) * torch.exp(2 * torch.randn((rows, 1), generator=gen))
    x[rows // 2] = 0
    x[rows // 3, cols - 1] = float("inf")
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_many_rows(cols, dtype):
    for rows in (613, 614, 615) if cols <= 2064 else (613,):
        check(values(rows, cols, dtype, rows + cols))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS + [65536, 65552])
def test_few_rows(cols, dtype):
    check(values(5, cols, dtype, cols))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(305, 65552), (1, 131056)])
def test_rows_longer_than_a_block_holds(rows, cols, dtype):
    check(values(rows, cols, dtype, 7))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(613, 16), (613, 272), (2503, 5376)])
def test_dequant(rows, cols, dtype):
    gen = torch.Generator().manual_seed(rows + cols)
    codes = torch.randint(-128, 128, (rows, cols), generator=gen, dtype=torch.int8)
    scale = torch.rand(rows, generator=gen) * 1e-2
    buf, y = guarded((rows, cols), dtype, -5.0)
    w4.int8_dequant(codes.cuda(), scale.cuda(), out=y)
    assert torch.equal(y.cpu(), (codes.float() * scale[:, None]).to(dtype)) and untouched(buf, -5.0)
