"""Host threads that share a stream, and therefore its workspace (or the library's
fixed scratch): the passes of one call are enqueued without another call's between
them (no GPU needed: the library is replaced by one that records when a call starts
and ends)."""
import threading
import time

import pytest
import torch

from exact_laplace_b200 import laplex as X


class Recorder:
    """Every laplex_* call records its start and its end, and sleeps between them
    (as a C call it would have given up the interpreter's lock)."""

    def __init__(self):
        self.log = []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            def size(*args):
                args[-1]._obj.value = 4096
                return X.OK
            return size

        def call(*args):
            me = threading.get_ident()
            self.log.append((me, "start"))
            time.sleep(0.02)
            self.log.append((me, "end"))
            return X.OK
        return call


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    ws = torch.zeros(8192, dtype=torch.uint8)
    monkeypatch.setattr(X, "lib", lambda: r)
    monkeypatch.setattr(X, "_seq_dev", lambda *ts: torch.device("cpu"))
    monkeypatch.setattr(X, "_dev", lambda *ts: torch.device("cpu"))
    monkeypatch.setattr(X, "_on", lambda dev: X._HERE_CTX)
    monkeypatch.setattr(X, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(X, "_stream", lambda dev: None)
    monkeypatch.setattr(X.Workspace, "get", classmethod(lambda cls, dev, nbytes: ws))
    monkeypatch.setattr(X, "_ws_sizes", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return r


def calls():
    x, lam = torch.zeros(40, 2, 8), torch.zeros(2)
    tok, g = torch.zeros(40, dtype=torch.int32), torch.zeros(40, 8)
    a = torch.zeros(40)
    p = torch.zeros(40, dtype=torch.int32)
    return {
        "linattn": lambda: X.linattn(x, x, x, lam),
        "linattn_backward": lambda: X.linattn_backward(x, x, x, lam, x),
        "embed_backward": lambda: X.embed_backward(tok, g, 5),
        "sort_anchors": lambda: X.sort_anchors(a),
        "sort_anchors_carry": lambda: X.sort_anchors_carry(a, a),
        "matvec_sym_unsorted": lambda: X.matvec_sym_unsorted(a, a),
        "matvec_sym": lambda: X.matvec_sym(a, a),
        "permute": lambda: X.permute(a, p),
        "invert_perm": lambda: X.invert_perm(p),
        "matvec_sym_planned": lambda: X.matvec_sym_planned(a, p, p, a),
        "matvec_general": lambda: X.matvec_general(a, a, a),
        "matvec_phased": lambda: X.matvec_phased(a, a, a),
        "gram": lambda: X.gram(a, a),
        "backward": lambda: X.backward(a, a, a),
        "backward_general": lambda: X.backward_general(a, a, a, a),
        "backward_phased": lambda: X.backward_phased(a, a, a, a),
        "gram_matrix": lambda: X.gram_matrix(a, a),
        "matvec_sym_noalloc": lambda: X.matvec_sym_noalloc(a, a),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_calls_of_two_threads_do_not_interleave(recorder, name):
    fns = calls()
    start = threading.Barrier(2)

    def run(fn):
        start.wait()
        fn()
        fn()

    ts = [threading.Thread(target=run, args=(fns[n],)) for n in (name, "embed_backward")]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert len(recorder.log) == 8
    for i in range(0, 8, 2):
        (a, x), (b, y) = recorder.log[i:i + 2]
        assert a == b and (x, y) == ("start", "end"), recorder.log


def test_a_refused_call_does_not_keep_the_others_waiting(recorder, monkeypatch):
    x = torch.zeros(40, 2, 8)
    with pytest.raises(X.LaplexError):
        X.linattn(x, x, x, torch.zeros(2), out=x[:3])
    monkeypatch.setattr(Recorder, "laplex_linattn", lambda self, *a: X.EINVAL, raising=False)
    monkeypatch.setattr(Recorder, "laplex_last_error", lambda self: b"refused", raising=False)
    with pytest.raises(X.LaplexError):
        X.linattn(x, x, x, torch.zeros(2))
    t = threading.Thread(target=calls()["embed_backward"], daemon=True)
    t.start()
    t.join(5)
    assert not t.is_alive()


def test_the_table_of_workspace_sizes_is_bounded(recorder, monkeypatch):
    monkeypatch.setattr(Recorder, "laplex_embed_backward", lambda self, *a: X.OK, raising=False)
    tok, g = torch.zeros(5000, dtype=torch.int32), torch.zeros(5000, 8)
    for n in range(1, 5000):
        X.embed_backward(tok[:n], g[:n], 3)
    assert 0 < len(X._ws_sizes) <= 4096
