"""The product's kernels right behind one another and behind other kernels: what a
block leaves behind in shared or tensor memory, or lets arrive there late, must not
reach the next one. Every result repeats the first bit for bit."""
import random

import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from test_gpu_int8_matmul import check, operands  # noqa: E402

pytestmark = pytest.mark.gpu

# whole tiles, clusters, shared units and pairs, few steps of K and many, one tile to a block and several
SHAPES = [(16, 2048, 16), (16, 4096, 2048), (40, 264, 4112), (64, 16384, 144), (64, 20488, 656), (12, 20488, 80),
          (128, 4104, 1040), (128, 20488, 272), (300, 2600, 528), (300, 10248, 144), (700, 4096, 272)]


def test_back_to_back():
    rng = random.Random(3)
    calls = [operands(*s, i) for i, s in enumerate(SHAPES)]
    want = [w4.int8_matmul(*c) for c in calls]
    for y, c in zip(want, calls):
        check(y, *c)
    r = torch.randn((40, 2608), device="cuda").bfloat16()
    weight = torch.ones(2608, device="cuda").bfloat16()
    _, codes, scale = w4.block_norm(r, weight, quantize=True)
    mx = w4.mxfp4_quantize(torch.randn((64, 1024), device="cuda").bfloat16(), 1)
    mx_y = w4.mxfp4_matmul(*mx, *mx)
    for _ in range(40):
        order = [rng.randrange(len(calls)) for _ in range(50)]
        got = []
        for i in order:
            got.append(w4.int8_matmul(*calls[i]))
            other = rng.randrange(4)
            if other == 0:
                assert torch.equal(w4.block_norm(r, weight, quantize=True)[1], codes)
            elif other == 1:
                assert torch.equal(w4.mxfp4_matmul(*mx, *mx), mx_y)
        for i, y in zip(order, got):
            assert torch.equal(y, want[i]), SHAPES[i]
    assert w4.device_status() == w4.OK
