"""The bounded waits of the tensor-core products and state passes: copies that
never come end in an error status, with nothing written outside the outputs, and
the next call is exact.  (The bound is short, and no copy is faulty: the first one
of each block is left out.)"""
import pytest
import torch

from exact_laplace_b200 import laplex as X
from test_gpu_linattn import DT, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,lens", [((2, 1, 64, 64), (200,)), ((4, 2, 128, 128), (2500, 0, 300)),
                                        ((2, 2, 72, 40), (90, 700)), ((8, 8, 64, 128), (400,) * 40)], ids=str)
def test_expired_waits(dt, heads, lens):
    c = Case(dt, lens, *heads, lam=[-0.1] * heads[1])
    want, grads = c.run_forward(), c.run_backward()
    t, pad = c.q.shape[0], 16
    whole = [torch.full((t + 2 * pad, *x.shape[1:]), 7.0, dtype=DT[dt], device="cuda") for x in (want[0], c.q, c.k, c.v)]
    inner = [x[pad:pad + t] for x in whole]
    for call in (lambda: c.run_forward(out=inner[0]), lambda: c.run_backward(out=tuple(inner[1:]))):
        X.device_status()
        X.test_set_linattn_wait(16, True)
        try:
            call()
        finally:
            X.test_set_linattn_wait()
        with pytest.raises(X.LaplexError) as e:
            X.device_status()
        assert e.value.status == X.ETIMEOUT
    assert all(bool((x[:pad] == 7).all()) and bool((x[pad + t:] == 7).all()) for x in whole)
    X.device_status()  # cleared after being reported
    assert all(torch.equal(a, b) for a, b in zip(c.run_forward(), want))
    assert all(torch.equal(a, b) for a, b in zip(c.run_backward()[:4], grads[:4]))


def test_expired_wait_in_a_replay():
    c = Case("bf16", (900, 30), 2, 1, 64, 64)
    want = c.run_forward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        good = c.run_forward()
        X.test_set_linattn_wait(16, True)
        try:
            c.run_forward()
        finally:
            X.test_set_linattn_wait()
        after = c.run_forward()
    X.device_status()
    graph.replay()
    with pytest.raises(X.LaplexError) as e:
        X.device_status()
    assert e.value.status == X.ETIMEOUT
    X.device_status()
    assert all(torch.equal(a, b) and torch.equal(d, b) for a, b, d in zip(good, want, after))
