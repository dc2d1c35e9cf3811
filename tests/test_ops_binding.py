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


def test_a_workspace_stays_where_it_is_when_its_object_is_used_on_another_gpu(monkeypatch):
    """Graphs captured on the first GPU hold its address."""
    made = []

    def on(stream, nbytes, device):
        made.append(types.SimpleNamespace(buffer=types.SimpleNamespace(device=device), address=256 * (len(made) + 1), use=lambda stream: None, nbytes=nbytes))
        return made[-1]

    monkeypatch.setattr(ops._Workspace, "on", on)
    monkeypatch.setattr(ops, "_here", lambda who, name, t: t.get_device())
    for op, call in ((ops.LayerNorm(64), lambda op, t: op.backward(t, t, None, t, t, t, dbias=t)), (ops.RMSNorm(64), lambda op, t: op.backward(t, t, t, t, t, dweight=t)),
                     (ops.ExpertRows(4, 2), lambda op, t: op.route(t, t, t, t))):
        made.clear()
        given = []
        for name, at in (("_backward", -3), ("_route", -3)):
            setattr(op, name, lambda *args, at=at: given.append(args[at]) or 0)
        monkeypatch.setattr(op, "_rows", lambda *a: (0, 0), raising=False)
        monkeypatch.setattr(op, "_flat", lambda *a: 0)
        for gpu in (0, 1, 0, 0, 1):
            call(op, types.SimpleNamespace(shape=(3, 2), device=gpu, dtype=None, get_device=lambda gpu=gpu: gpu, element_size=lambda: 4))
        assert given == [256, 512, 256, 256, 512] and len(made) == 2 and made[0].nbytes == op.workspace_bytes
