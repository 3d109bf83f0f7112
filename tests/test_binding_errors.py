"""A call that the library refuses raises, with the status and the entry point's own name:
every operator of the int8 rows and the block norm. Stand-in tensors, and a library that
answers as it is told (no device needed)."""
import pytest

import weight_only_int4_gb300 as w4

torch = pytest.importorskip("torch")
from test_binding_checks import Library, Tensor, operands  # noqa: E402
from test_binding_int8 import CALLS, outputs  # noqa: E402


class Refusing(Library):
    def __init__(self, status):
        super().__init__()
        self.status = status

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("workspace_bytes"):
                return 4096
            self.launched.append(name)
            return self.status
        return entry


@pytest.mark.parametrize("status", [w4.ERR_SHAPE, w4.ERR_ALIGN, w4.ERR_WORKSPACE, w4.ERR_CUDA])
@pytest.mark.parametrize("name", list(CALLS))
def test_refused(name, status, monkeypatch):
    w4._torch()
    lib = Refusing(status)
    monkeypatch.setattr(w4, "load_library", lambda: lib)
    monkeypatch.setattr(w4, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(w4, "_stream_ptr", lambda stream=None: 0)
    call, spec, outs, takes_workspace = CALLS[name]
    kw = dict(workspace=Tensor((1 << 20,), torch.uint8)) if takes_workspace else {}
    entry = "w4a16_" + name.split(",")[0]
    with pytest.raises(w4.W4A16Error, match=f"^{entry} failed: {w4.STATUS_NAMES[status]}$") as e:
        call(operands(spec), out=outputs(outs), **kw)
    assert e.value.status == status and lib.launched == [entry]
