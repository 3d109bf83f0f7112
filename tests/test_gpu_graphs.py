"""CUDA graphs captured through calls that bring no workspace, with no eager call
of the same kind before: each graph has to carry the zero fill that its kernels
rely on, whichever is replayed first. Results are compared bit for bit with
calls on a workspace of the test's own.
"""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from gpu_util import DeviceCase  # noqa: E402
from w4a16_inputs import make_case  # noqa: E402

pytestmark = pytest.mark.gpu


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def words(gen, *shape):
    return torch.randint(-2 ** 31, 2 ** 31, shape, dtype=torch.int32, device="cuda", generator=gen)


def scales(gen, *shape):
    return torch.randint(118, 122, shape, dtype=torch.uint8, device="cuda", generator=gen)


def moe_call(T, seed, E=16, k=4, H=512, I=256):
    gen = generator(seed)
    x = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    router = (torch.randn((E, H), device="cuda", generator=gen) / H ** 0.5).bfloat16()
    args = (x, router, words(gen, E, H // 8, 2 * I), scales(gen, E, H // 32, 2 * I), words(gen, E, I // 8, H),
            scales(gen, E, I // 32, H), k)
    need = w4.load_library().w4a16_mxfp4_moe_workspace_bytes(T, E, k, H, I)
    return lambda **kw: w4.mxfp4_moe(*args, **kw), need


def product_call(M, N, seed, K=512):
    """More column tiles than SMs, few rows: tiles shared between thread blocks, joined by tickets."""
    gen = generator(seed)
    args = (words(gen, M, K // 8), w4.mxfp4_tile_scales(scales(gen, M, K // 32)), words(gen, N, K // 8),
            w4.mxfp4_tile_scales(scales(gen, N, K // 32)))
    return lambda **kw: w4.mxfp4_matmul(*args, **kw), w4.workspace_bytes(w4.OP_MXFP4_MATMUL, M, N, K, 32)


def gemv_call(M, N, seed, K=512, g=32):
    """Stream-K with tickets."""
    dc = DeviceCase(make_case(M, N, K, g, "f16", False, seed=seed))
    return (lambda **kw: w4.gemv(dc.x, dc.qw, dc.s, dc.qz, g, **kw)), w4.workspace_bytes(w4.OP_GEMV, M, N, K, g)


PAIRS = {
    "moe": (lambda: moe_call(40, 1), lambda: moe_call(2, 2)),
    "product": (lambda: product_call(16, 24576, 3), lambda: product_call(9, 20480, 4)),
    "gemv": (lambda: gemv_call(3, 24576, 5), lambda: gemv_call(3, 20480, 6)),
}


@pytest.mark.parametrize("kind", list(PAIRS))
def test_two_graphs_captured_cold(kind):
    """The larger call captured first, the smaller one replayed first, then both in turn."""
    calls = [make() for make in PAIRS[kind]]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graphs, outs = [], []
    for call, _ in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(call())
        graphs.append(graph)
    want = [call(workspace=w4.new_workspace(need)) for call, need in calls]
    torch.cuda.synchronize()
    for i in (1, 1, 0, 1, 0, 0, 1):
        outs[i].zero_()
        torch.cuda.synchronize()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
    assert w4.device_status() == w4.OK


@pytest.mark.parametrize("op", [w4.OP_GEMV, w4.OP_GEMM])
def test_tickets_lie_where_the_fill_of_a_capture_begins(op):
    """The smallest shape needs one rounded-up group of ticket words after the partial sums."""
    need = w4.workspace_bytes(op, 1, 8, 32, 32)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert w4._zero_range(op, need, sms) == (need - 256, need)


def test_capture_id():
    lib = w4.load_library()
    stream = torch.cuda.Stream()
    seen = []
    for _ in range(2):
        assert lib.w4a16_capture_id(stream.cuda_stream) == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            first, again = (lib.w4a16_capture_id(stream.cuda_stream) for _ in range(2))
            torch.zeros(4, device="cuda").add_(1)
        assert first == again != 0
        seen.append(first)
    assert seen[0] != seen[1]
    assert lib.w4a16_capture_id(stream.cuda_stream) == 0
