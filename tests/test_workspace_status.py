"""The binding's workspaces keep the device status (no GPU needed: CPU memory
stands in for the device's)."""
import types

import pytest
import torch

from exact_laplace_b200 import laplex as X


@pytest.fixture
def cache(monkeypatch):
    monkeypatch.setattr(X.Workspace, "_cache", {})
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def test_a_larger_workspace_takes_the_status_along(cache):
    dev = torch.device("cpu")
    ws = X.Workspace.get(dev, 1000)
    assert not ws.any()
    ws[0] = 2  # a call recorded LAPLEX_ETIMEOUT
    ws[256:] = 9
    assert X.Workspace.get(dev, 500) is ws
    larger = X.Workspace.get(dev, 5000)
    assert larger.numel() >= 5000 and larger[0] == 2 and not larger[1:].any()
