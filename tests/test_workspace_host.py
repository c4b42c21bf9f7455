"""The cached workspaces on the host (no GPU): torch's stream calls are replaced."""
import types
import weakref

import pytest
import torch

import w4_gemm_gated_amd as sp
from w4_gemm_gated_amd import serve


@pytest.fixture
def stream(monkeypatch):
    s = types.SimpleNamespace(cuda_stream=5, capturing=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: s)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s.capturing)
    monkeypatch.setattr(sp, "_workspaces", {})
    if hasattr(sp, "_replaced_workspaces"):
        monkeypatch.setattr(sp, "_replaced_workspaces", [])
    return s


def test_a_replaced_workspace_stays_alive(stream):
    """A graph captured with it holds its address."""
    first = sp._workspace(1000, "cpu")
    at, alive = first.data_ptr(), weakref.ref(first)
    assert sp._workspace(1 << 20, "cpu") is first
    del first
    larger = sp._workspace((1 << 20) + 1, "cpu")
    assert larger.numel() > 1 << 20 and not larger.any()
    assert alive() is not None and alive().data_ptr() == at
    assert serve._scratch(1 << 20, torch.device("cpu"), 5) is larger


def test_replaced_workspaces_stay_small(stream):
    for n in range(1 << 20, 9 << 20, 123457):
        ws = sp._workspace(n, "cpu")
    assert sum(w.numel() for w in sp._replaced_workspaces) <= ws.numel()


def test_capture_needs_a_workspace_that_is_there(stream):
    stream.capturing = True
    for need in (sp._workspace, lambda n, d: serve._scratch(n, torch.device(d), 5)):
        with pytest.raises(RuntimeError, match="workspace="):
            need(4096, "cpu")
    assert not sp._workspaces
    assert sp._workspace(0, "cpu") is None
    stream.capturing = False
    ws = sp._workspace(4096, "cpu")
    stream.capturing = True
    assert sp._workspace(4096, "cpu") is ws
    with pytest.raises(RuntimeError, match="workspace="):
        sp._workspace((1 << 20) + 1, "cpu")
    stream.cuda_stream = 6                      # another stream has none
    with pytest.raises(RuntimeError, match="workspace="):
        sp._workspace(4096, "cpu")
