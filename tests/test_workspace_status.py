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


class Library:
    def __init__(self):
        self.log = []

    def laplex_set_status_word(self, p):
        self.log.append(("word", p))
        return X.OK

    def laplex_workspace_init(self, p, n, stream):
        self.log.append(("init", p, stream))
        return X.OK

    def laplex_embed_backward_workspace_size(self, *args):
        args[-1]._obj.value = 512
        return X.OK

    def laplex_embed_backward(self, *args):
        self.log.append(("call",))
        return X.EINVAL if self.fail else X.OK

    def laplex_get_device_status(self, p, stream):
        self.log.append(("status", p.value))
        return X.OK

    def laplex_last_error(self):
        return b"refused"

    fail = False


@pytest.mark.parametrize("fail", [False, True])
def test_a_captured_call_reports_outside_the_graphs_memory(cache, monkeypatch, fail):
    lib, dev = Library(), torch.device("cpu")
    lib.fail = fail
    streams = iter([types.SimpleNamespace(cuda_stream=i) for i in (5, 6)])
    monkeypatch.setattr(X, "lib", lambda: lib)
    monkeypatch.setattr(X.Workspace, "_words", {})
    monkeypatch.setattr(X, "_seq_dev", lambda *ts: dev)
    monkeypatch.setattr(X, "_on", lambda d: X._HERE_CTX)
    monkeypatch.setattr(X, "_raw_stream", lambda d: 5)
    monkeypatch.setattr(X, "_stream", lambda d: None)
    monkeypatch.setattr(X, "_ws_sizes", {})
    monkeypatch.setattr(X, "_capturing", lambda s: s.cuda_stream == 5)
    monkeypatch.setattr(torch.cuda, "Stream", lambda d: next(streams))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d: lib.log.append(("synchronize",)))
    tok, g = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)
    for _ in range(2):
        if fail:
            with pytest.raises(X.LaplexError):
                X.embed_backward(tok, g, 3)
        else:
            X.embed_backward(tok, g, 3)
    word = X.Workspace._words[dev]
    one = [("word", word.data_ptr()), ("call",), ("word", None)]
    # cleared once, on a stream that is not captured
    assert lib.log == [("init", word.data_ptr(), 6)] + 2 * one
    lib.log.clear()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    X.device_status(dev)
    assert lib.log == [("synchronize",), ("status", word.data_ptr())]
