"""The operators' Python side, on the CPU: its bookkeeping of streams, against stand-ins for torch's."""
import sys
import types

from conftest import ensure_built

ensure_built()

from device_triggered_transfers_gb300 import ops  # noqa: E402


def stand_in(recorded):
    """The little of torch that a workspace asks for; a buffer keeps the streams it was recorded on."""
    stream = types.SimpleNamespace(synchronize=lambda: None)
    buffer = types.SimpleNamespace(device="device", data_ptr=lambda: 256, record_stream=recorded.append)
    cuda = types.SimpleNamespace(current_stream=lambda device: stream, default_stream=lambda device: "default",
                                 ExternalStream=lambda address, device: ("external", address))
    return types.SimpleNamespace(uint8=None, cuda=cuda, empty=lambda nbytes, dtype, device: buffer)


def test_every_stream_that_uses_a_workspace_is_recorded_the_default_one_too(monkeypatch):
    recorded = []
    monkeypatch.setitem(sys.modules, "torch", stand_in(recorded))
    w = ops._Workspace(64, "device")
    side = object()
    for stream in (None, None, side, side, None, 77, None):
        w.use(stream)
    assert recorded == ["default", side, "default", ("external", 77), "default"]
