"""A workspace is made and read with its own device current, and only on a GPU.
The library and the devices are stand-ins here: no GPU."""
import contextlib

import pytest
import torch

import rank_markov_draft_amd as rmd
from rank_markov_draft_amd import _lib


@pytest.mark.parametrize("device", ["cpu", "meta", torch.device("cpu")])
def test_workspace_off_the_gpu_is_refused(device):
    """Before its memory is handed to a kernel."""
    with pytest.raises(ValueError, match="runs on a GPU"):
        rmd.Workspace(2, 3, 64, 16, sample=True, device=device)


@pytest.fixture
def two_devices(monkeypatch):
    """Calls of the library as (name, current device, stream); device 0 is current."""
    current, calls = [0], []

    @contextlib.contextmanager
    def use(device):
        before, current[0] = current[0], torch.device(device).index
        yield
        current[0] = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 4096
                calls.append((name, current[0], args[2] if name.endswith("init") else args[1]))
                return 0
            return call

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw))
    monkeypatch.setattr(rmd, "_stream_handle", lambda device: ("stream of", device.index))
    monkeypatch.setattr(_lib, "load", Library)
    return calls


@pytest.mark.parametrize("device,index", [(None, 0), ("cuda", 0), ("cuda:0", 0), ("cuda:1", 1), (torch.device("cuda", 1), 1)])
def test_workspace_is_made_and_read_on_its_device(two_devices, device, index):
    ws = rmd.Workspace(2, 3, 64, 16, sample=True, processed=True, device=device)
    assert two_devices == [("dspark_markov_workspace_init", index, ("stream of", index))]
    del two_devices[:]
    rmd.read_device_error(ws)
    assert two_devices == [("dspark_markov_read_device_error", index, ("stream of", index))]
