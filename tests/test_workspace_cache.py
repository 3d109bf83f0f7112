"""The binding's own workspaces, on the CPU: which calls share one.

Streams, tensors and the capture query are stand-ins; what is checked is the
binding's bookkeeping alone.
"""
import contextlib
import types

import pytest

import weight_only_int4_gb300 as w4


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Device:
    index = 0


@pytest.fixture
def world(monkeypatch):
    """A stand-in for the library and torch; `capture` maps a stream handle to the capture that it is in."""
    capture = {}
    made = []

    def new_workspace(nbytes, device=None):
        made.append(types.SimpleNamespace(numel=lambda n=nbytes: n))
        return made[-1]

    cuda = types.SimpleNamespace(stream=lambda s: contextlib.nullcontext(), current_device=lambda: 0,
                                 get_device_properties=lambda d: types.SimpleNamespace(multi_processor_count=152))
    monkeypatch.setattr(w4, "_torch", lambda: types.SimpleNamespace(cuda=cuda))
    monkeypatch.setattr(w4, "load_library",
                        lambda: types.SimpleNamespace(w4a16_capture_id=lambda handle: capture.get(handle, 0)))
    monkeypatch.setattr(w4, "new_workspace", new_workspace)
    monkeypatch.setattr(w4, "_captured_workspace", lambda nbytes, device, op, sms: new_workspace(nbytes),
                        raising=False)
    monkeypatch.setattr(w4, "_workspaces", {})
    monkeypatch.setattr(w4, "_retired", [])
    return types.SimpleNamespace(capture=capture, made=made,
                                 get=lambda s, n=100, op=w4.OP_GEMV: w4._cached_workspace(n, Device, s, op))


def test_eager_calls_on_a_stream_share_one(world):
    a, b = Stream(1), Stream(2)
    first = world.get(a)
    assert world.get(a, 60) is first
    assert world.get(b) is not first
    assert world.get(a, op=w4.OP_GEMM) is not first
    grown = world.get(a, 300)
    assert grown is not first and world.get(a) is grown
    assert first in w4._retired


def test_each_capture_has_its_own(world):
    """The zero fill of a workspace made during a capture belongs to that graph: a second capture on the same
    stream, of the same or a smaller shape, cannot rely on it."""
    s = Stream(7)
    world.capture[7] = 41
    large = world.get(s, 500)
    assert world.get(s, 200) is large                 # one capture: one workspace
    world.capture[7] = 42
    small = world.get(s, 200)
    assert small is not large
    assert world.get(s, 200) is small
    del world.capture[7]
    eager = world.get(s, 200)
    assert eager is not large and eager is not small  # no graph's fill serves an eager call
    world.capture[7] = 43
    assert world.get(s, 200) is not eager             # and a graph does not run in the eager calls' memory
    kept = list(w4._workspaces.values()) + w4._retired
    assert all(any(m is k for k in kept) for m in world.made)   # graphs may replay: nothing was dropped
    w4.release_workspaces()
    assert not w4._workspaces and not w4._retired


@pytest.mark.parametrize("op", [w4.OP_GEMV, w4.OP_GEMM, w4.OP_MXFP4_MATMUL, "mxfp4_moe"])
@pytest.mark.parametrize("nbytes", [256, 1 << 20, 50 << 20])
def test_captured_fill_covers_what_must_start_at_zero(op, nbytes):
    """Ticket words after the partial sums (everything where there are none), or barrier words at the start."""
    torch = pytest.importorskip("torch")
    first, last = w4._zero_range(op, nbytes, 152)
    if op == "mxfp4_moe":
        assert (first, last) == (0, 256)
    else:
        partials = 152 * (136 if op == w4.OP_GEMV else 128) * 1024
        assert (first, last) == ((partials if nbytes > partials else 0), nbytes)
    ws = w4._captured_workspace(nbytes, torch.device("cpu"), op, 152)
    assert ws.numel() == nbytes and not ws[first:last].any()


def test_a_failed_size_query_is_not_remembered(monkeypatch):
    """The library answers 0 where no GB300 is current: the next call of the shape asks again."""
    answers = [0, 4096, 8192]
    ws = types.SimpleNamespace(data_ptr=lambda: 0x10000, numel=lambda: 4096, element_size=lambda: 1)
    monkeypatch.setattr(w4, "_workspace_needs", {})
    monkeypatch.setattr(w4, "_cached_workspace", lambda nbytes, device, stream, op: ws)
    ask = lambda: w4._workspace(None, "op", lambda *shape: answers.pop(0), (1, 2, 3), Device, None)
    assert ask() == (0, 0)
    assert ask() == (0x10000, 4096)
    assert ask() == (0x10000, 4096) and answers == [8192]   # a size is
