"""The example block (quantise, product, experts) and its CUDA graph.

Tolerance: the block's output and its FP32 form share every operand and the
rounding of the projection; what differs is bf16 rounding of the experts' sum
and of the output (2^-8 each) and the experts' own error (below 2^-9 of sums
that stay below the largest output here): under 1.6e-2 of the largest output,
the bound of the bf16 layers.
"""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 8, 40])
def test_example(tokens):
    import mxfp4_moe_block as ex
    assert ex.main(tokens) <= 1.6e-2


def test_block_in_a_graph():
    import mxfp4_moe_block as ex
    block = ex.MoeBlock(hidden=512, inner=256, experts=8, top_k=2)
    x = torch.randn((5, 512), device="cuda").to(torch.bfloat16)
    ref = block(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, block(x))
