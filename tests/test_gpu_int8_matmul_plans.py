"""The int8 product in every way that it runs a shape, each named in test_int8_plan.py,
against 64-bit arithmetic, and again bit for bit. A row in the last of many chunks too."""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from test_gpu_int8_matmul import run  # noqa: E402
from test_int8_plan import PLANS  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", list(PLANS))
def test_every_way(M, N, K, dtype):
    a, sa, b, sb, y = run(M, N, K, dtype)
    for _ in range(2):
        assert torch.equal(w4.int8_matmul(a, sa, b, sb, out_dtype=dtype), y)
    assert w4.device_status() == w4.OK
    w4.release_workspaces()
