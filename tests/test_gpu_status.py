"""Device errors reach device_status() whatever became of the workspace that the
call ran in: replaced by a larger one, or memory of a captured graph."""
import pytest
import torch

from exact_laplace_b200 import laplex as X

pytestmark = pytest.mark.gpu


def test_status_of_a_replaced_workspace():
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = torch.randn(5000, device="cuda")
        a[7] = float("nan")
        X.sort_anchors(a)
        before = X.Workspace.get(a.device, 0)
        tok = torch.randint(0, 50, (400000,), device="cuda")
        X.embed_backward(tok, torch.randn(400000, 8, device="cuda"), 50)
        assert X.Workspace.get(a.device, 0) is not before
        with pytest.raises(X.LaplexError) as e:
            X.device_status()
        assert e.value.status == X.ENONFINITE
        X.device_status()  # cleared after being reported


@pytest.mark.parametrize("known", [False, True])
def test_status_of_a_captured_call(monkeypatch, known):
    """An expired wait in a replay, with the graph's workspace taken over by its later
    calls; with and without the device's word there before the capture."""
    if not known:
        monkeypatch.setattr(X.Workspace, "_words", {})
    n, rows = 70000, 900
    t = torch.randint(0, rows, (n,), device="cuda")
    g = torch.randn(n, 8, device="cuda")
    want = X.embed_backward(t, g, rows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        good = X.embed_backward(t, g, rows)
        X.test_set_sort_wait(16, True)
        try:
            X.embed_backward(t, g, rows)
        finally:
            X.test_set_sort_wait()
        more = [torch.ones(100000, device="cuda") for _ in range(40)]
        after = X.embed_backward(t, g, rows)
    X.device_status()  # nothing ran
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        with torch.cuda.stream(side):
            graph.replay()
        with pytest.raises(X.LaplexError) as e:
            X.device_status()
        assert e.value.status == X.ETIMEOUT
        assert torch.equal(good, want) and torch.equal(after, want)
    X.device_status()
    assert all(bool((x == 1).all()) for x in more)
    X.embed_backward(t, g, rows)  # an eager call reports to its stream's workspace again
    X.device_status()


def test_the_word_is_aligned():
    assert X.lib().laplex_set_status_word(258) == X.EINVAL
    assert X.lib().laplex_set_status_word(None) == X.OK
