"""The int8 operators and the block norm together: the example block runs, agrees
with the same block in FP32 on the dense copies, alone and in a captured graph.

Tolerance, as a share of the largest output: what the two forms do differently is
FP32 arithmetic, which moves values across rounding borders. One bfloat16 value on
another side of a border moves by 2^-8 of itself, one code by one step of 127. A sum of
1024 or 2048 products of which a few in a thousand move that far is off by far less than
such a step; two steps of bfloat16 and one of int8 bound the output: 2 * 2^-8 + 1 / 127.
"""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import int8_block  # noqa: E402

pytestmark = pytest.mark.gpu

TOL = 2 * 2.0 ** -8 + 1 / 127


@pytest.mark.parametrize("tokens", [1, 8, 100, 300])
def test_example(tokens):
    assert int8_block.main(tokens) <= TOL


def test_two_blocks_in_a_graph():
    """Two blocks in turn, captured cold, replayed on new inputs: the same bits as the calls by themselves."""
    first, second = int8_block.Int8Block(512, 272, seed=1), int8_block.Int8Block(512, 272, seed=2)
    r = torch.randn((37, 512), device="cuda")

    def step(x):
        y, _ = first(x)
        return second(y)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(r)
    for seed in (3, 4, 3):
        r.copy_(torch.randn((37, 512), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        want = step(r)
        torch.cuda.synchronize()
        assert all(torch.equal(g, x) for g, x in zip(out, want))
    assert w4.device_status() == w4.OK


def test_another_stream():
    """The whole block on a stream of its own, given to every call's surroundings."""
    block = int8_block.Int8Block(1040, 528, seed=5)
    r = torch.randn((19, 1040), device="cuda")
    want = block(r)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = block(r)
    stream.synchronize()
    assert all(torch.equal(g, x) for g, x in zip(got, want))


def test_streams_as_arguments():
    """stream= of each call: outputs belong to it, results are the same."""
    stream = torch.cuda.Stream()
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((33, 528), device="cuda", generator=gen).bfloat16()
    w = w4.int8_quantize(torch.randn((264, 528), device="cuda", generator=gen))
    ones = torch.ones(528, device="cuda").bfloat16()
    torch.cuda.synchronize()
    c, s = w4.int8_quantize(x, stream=stream)
    y = w4.int8_matmul(c, s, *w, stream=stream)
    d = w4.int8_dequant(c, s, stream=stream)
    n = w4.block_norm(x, ones, x, quantize=True, stream=stream)
    stream.synchronize()
    want = w4.int8_quantize(x)
    assert torch.equal(c, want[0]) and torch.equal(s, want[1])
    assert torch.equal(y, w4.int8_matmul(*want, *w)) and torch.equal(d, w4.int8_dequant(*want))
    assert all(torch.equal(a, b) for a, b in zip(n, w4.block_norm(x, ones, x, quantize=True)))
