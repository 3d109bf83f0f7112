"""How far a sum is exact: as long as sum |a b| does not exceed 2^24, whatever K and
whichever kernel runs. Past that few rows stay exact in 32 bits, and all stay within the
bound of test_gpu_int8_matmul.py."""
import math

import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from test_gpu_int8_matmul import check  # noqa: E402

pytestmark = pytest.mark.gpu

# dot products, tiles of 16 to 128 rows, pairs
ROWS = [1, 4, 8, 40, 128, 300]


def one(n):
    return torch.ones(n, device="cuda")


@pytest.mark.parametrize("K", [2064, 5376, 21504, 131056])
@pytest.mark.parametrize("M", ROWS)
def test_up_to_the_limit(M, K):
    """Codes of one sign, as large as K lets them be, and neighbours that make the sum odd."""
    N, c = 264, math.isqrt(2 ** 24 // K)
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    a = torch.full((M, K), c, dtype=torch.int8, device="cuda")
    b = torch.full((N, K), c, dtype=torch.int8, device="cuda")
    a -= torch.randint(0, 2, (M, K), device="cuda", generator=gen).to(torch.int8)
    b -= torch.randint(0, 2, (N, K), device="cuda", generator=gen).to(torch.int8)
    b[1::2] *= -1
    want = a.double() @ b.double().T
    assert bool((want.abs() <= 2.0 ** 24).all())
    assert torch.equal(w4.int8_matmul(a, one(M), b, one(N), out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("K", [5376, 131056])
@pytest.mark.parametrize("M", ROWS)
def test_past_the_limit(M, K):
    N = 264
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    a = torch.randint(0, 128, (M, K), device="cuda", generator=gen).to(torch.int8)
    b = torch.randint(0, 128, (N, K), device="cuda", generator=gen).to(torch.int8)
    y = w4.int8_matmul(a, one(M), b, one(N), out_dtype=torch.float32)
    check(y, a, one(M), b, one(N))
    if M <= 4:
        assert torch.equal(y, (a.double() @ b.double().T).float())
