"""Scales of the int8 product that are not ordinary numbers: y = (S sa) sb with S a whole
number, each product as FP32 gives it, so an infinity times a sum of zero is NaN."""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from test_gpu_int8_matmul import operands  # noqa: E402

pytestmark = pytest.mark.gpu


# dot products; tiles in clusters, whole, shared; pairs, and pairs with columns cut off
@pytest.mark.parametrize("M,N,K", [(1, 136, 272), (8, 136, 272), (40, 136, 272), (9, 1640, 1040), (16, 20488, 272),
                                   (128, 20488, 144), (300, 2600, 272), (700, 4096, 272), (201, 20000, 2368)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_as_the_products_give_it(M, N, K, dtype):
    a, sa, b, sb = operands(M, N, K, 9)
    a[M // 2] = 0                         # its sums are zero
    sa[0], sb[1], sb[2], sb[3] = float("inf"), float("-inf"), 0.0, float("nan")
    sb[N - 1], sb[N - 2] = 3e38, 1e-45
    if M > 2:
        sa[M - 1], sa[M - 2] = float("nan"), -2.0
    S = (a.double() @ b.double().T).float()   # whole numbers below 2^24
    want = ((S * sa[:, None]) * sb).to(dtype)
    y = w4.int8_matmul(a, sa, b, sb, out_dtype=dtype)
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.nan_to_num(nan=0.0, posinf=7.0, neginf=-7.0), want.nan_to_num(nan=0.0, posinf=7.0, neginf=-7.0))
    assert bool(y.isnan().any()) and (M == 1 or bool(y.isinf().any()))   # one row alone: the zero one
