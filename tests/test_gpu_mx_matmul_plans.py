"""The MXFP4 product on a shape of every plan, for every output type: 128-row
tiles over several K steps and tiles, tiles shared over a long ragged K, K
split over clusters. Bounds and operands as in the product's own tests; which
plan a shape takes is asserted on the host."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from test_gpu_mx_matmul import ULP, Operand, check  # noqa: E402
from test_mx_plan import PLANS, SMS, plan  # noqa: E402

pytestmark = pytest.mark.gpu


def test_the_plans_are_this_devices():
    assert torch.cuda.get_device_properties(0).multi_processor_count == SMS


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("shape", list(PLANS))
def test_plan(shape, dtype):
    M, N, K = shape
    check(Operand(M, K, M + N), Operand(N, K, M + K), dtype, shape)


@pytest.mark.parametrize("M,N,K,want", [(100, 12008, 2080, (128, 1, 0)), (300, 5128, 2080, (128, 1, 0)),
                                        (20, 20488, 2080, (32, 1, 1)), (90, 2600, 2080, (64, 1, 0))])
def test_each_block_has_its_own_exponent(M, N, K, want):
    """One-hot rows of A pick single elements of B: exact, whatever block, row tile and step they are in."""
    assert plan(w4.load_library(), M, N, K) == want
    B = Operand(N, K, 9, 100, 140)
    codes = np.zeros((M, K), dtype=np.uint8)
    cols = [(37 * m + 5) % K for m in range(M)]
    codes[np.arange(M), cols] = 2                      # 1.0
    A = Operand(M, K, 10, 127, 127)
    A.codes = codes
    A.e = (127 + (np.arange(M)[:, None] + np.arange(K // 32)[None, :]) % 5).astype(np.uint8)
    y = w4.mxfp4_matmul(*A.device(), *B.device(), out_dtype=torch.float32)
    scale = np.ldexp(1.0, A.e[np.arange(M), np.array(cols) // 32].astype(int) - 127)
    assert torch.equal(y.double(), B.values()[:, cols].T * torch.from_numpy(scale).cuda()[:, None])
