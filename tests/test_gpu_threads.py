"""Host threads that share one stream and its workspace: the same bits as one
thread alone."""
import threading

import pytest
import torch

from exact_laplace_b200 import laplex as X

pytestmark = pytest.mark.gpu


def work(seed):
    """Calls whose passes meet in the workspace, with their results of before."""
    g = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    q, k, v, do = (normal(2600, 2, 64).bfloat16() for _ in range(4))
    f = normal(1500, 2, 24)
    lam = torch.tensor([-0.01, -0.2], device="cuda")
    tok = torch.randint(0, 900, (5000,), generator=g, device="cuda")
    many = torch.randint(0, 5000, (70000,), generator=g, device="cuda")
    rows, wide = normal(5000, 72), normal(70000, 8)
    a = normal(30000)
    fns = [lambda: X.linattn(q, k, v, lam, return_state=True), lambda: X.linattn_backward(q, k, v, lam, do)[:3],
           lambda: X.linattn_backward(f, f, f, lam, f, return_dlog_decay=True)[:3],
           lambda: (X.embed_backward(tok, rows, 900),), lambda: (X.embed_backward(many, wide, 5000),),
           lambda: X.sort_anchors(a)]
    return [(fn, [x.clone() for x in fn()]) for fn in fns]


def test_threads_on_one_stream():
    todo = [work(seed) for seed in (1, 2, 3)]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(todo))

    def run(calls):
        try:
            start.wait()
            for _ in range(15):
                got = [(fn(), want) for fn, want in calls]
                for i, (res, want) in enumerate(got):
                    if not all(torch.equal(x, y) for x, y in zip(res, want)):
                        wrong.append(i)
        except Exception as e:  # (an assertion in a thread would not reach pytest)
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(calls,)) for calls in todo]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    X.device_status()
