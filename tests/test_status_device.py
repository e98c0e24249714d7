"""status() waits for a stream of the handle's device, whichever device is current (fakes stand for the devices)."""
import types

import torch

from speculative_decoding_tree_05_gb300 import ddtree


class FakeLibrary:
    def __init__(self, devices):
        self.devices, self.calls = devices, []

    def ddtree_read_device_status(self, workspace, out, stream):
        self.calls.append((self.devices[-1], stream.value))
        out._obj.value = 5
        return 0


def fake_devices(monkeypatch):
    """Device 0 is current; device i's current stream has the handle 1000 + i.  Returns the stack of current devices."""
    devices = [0]

    class Switch:
        def __init__(self, d):
            self.index = d.index if isinstance(d, torch.device) else d

        def __enter__(self):
            devices.append(self.index)

        def __exit__(self, *exc):
            devices.pop()

    def current_stream(d=None):
        index = devices[-1] if d is None else (d.index if isinstance(d, torch.device) else d)
        return types.SimpleNamespace(cuda_stream=1000 + index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: devices[-1])
    monkeypatch.setattr(torch.cuda, "device", Switch)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    return devices


def workspace_on(index):
    return types.SimpleNamespace(device=torch.device("cuda", index), data_ptr=lambda: 0x10000)


def test_the_workspaces_device(monkeypatch):
    library = FakeLibrary(fake_devices(monkeypatch))
    assert ddtree.read_device_status(workspace_on(1), library=library) == 5
    assert ddtree.read_device_status(workspace_on(0), library=library) == 5
    assert library.calls == [(1, 1001), (0, 1000)]


def test_a_given_stream(monkeypatch):
    library = FakeLibrary(fake_devices(monkeypatch))
    s = types.SimpleNamespace(cuda_stream=77)
    ddtree.read_device_status(workspace_on(1), s, library=library)
    assert library.calls == [(1, 77)]


def test_every_handle(monkeypatch):
    for cls in (ddtree.Verifier, ddtree.SparseVerifier, ddtree.KeyWeights, ddtree.BlockSelector, ddtree.BlockVerifier):
        with monkeypatch.context() as m:
            library = FakeLibrary(fake_devices(m))
            h = cls.__new__(cls)
            h.lib, h.workspace, h.device = library, workspace_on(1), torch.device("cuda", 1)
            assert h.status() == 5
            assert library.calls == [(1, 1001)], cls
