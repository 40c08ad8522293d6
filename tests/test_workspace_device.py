"""A layer's workspace is memory of one device: a call on another one is refused, though the streams' handles are the same
(the default stream's is 0 on every device).  No GPU: devices and streams are made up."""
import pytest

torch = pytest.importorskip("torch")

from transformer_head_scaled_02_gb300 import Mha  # noqa: E402
from transformer_head_scaled_02_gb300 import mha as front  # noqa: E402


class _On:
    """What the checks ask of a tensor on a device."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device

    def numel(self):
        return 1 << 20

    def record_stream(self, stream):
        pass


@pytest.fixture
def layer(monkeypatch):
    import __graft_entry__ as g
    g.build_library()
    now = [0]
    for name in ("_current_device", "_current_stream", "_capturing"):
        monkeypatch.setattr(front, name, {"_current_device": lambda: now[0]}.get(name, lambda *a: 0))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x = Mha(64, 1, 64, dtype=torch.float32, device="cpu")
    x.now = now
    monkeypatch.setattr(x, "_new_workspace", lambda nbytes: (_On(now[0]), 0))
    x.ensure_workspace(0, 0, 0, need=256)
    return x


def test_steps_on_the_workspace_s_device(layer):
    layer.ensure_workspace(0, 0, 0, need=1024)
    layer._hold_status()
    cache = type("Cache", (), {"_data": _On(0)})
    assert layer._quant_ready(cache, _On(0), _On(0), _On(0), None, 1024) == 0


def test_steps_on_another_device_are_refused(layer):
    layer.now[0] = 1
    with pytest.raises(ValueError, match="cuda:0"):
        layer.ensure_workspace(0, 0, 0, need=1024)
    with pytest.raises(ValueError, match="cuda:0"):
        layer._hold_status()
    cache = type("Cache", (), {"_data": _On(1)})
    with pytest.raises(ValueError, match="cuda:0"):
        layer._quant_ready(cache, _On(1), _On(1), _On(1), None, 1024)
