"""The table's gradient after a sort whose wait ran out: an error status, and no
access outside the call's arrays whatever the workspace held before."""
import pytest
import torch

from exact_laplace_b200 import laplex as X

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("dim", [8, 13])
@pytest.mark.parametrize("old", [0x00, 0x03, 0x7f, 0xff])
def test_expired_sort_stays_inside(dt, dim, old):
    n, rows, pad = 70000, 900, 64  # (more tokens than the one-cluster sort takes)
    t = torch.randint(0, rows, (n,), generator=torch.Generator().manual_seed(1)).cuda()
    g = torch.randn(n, dim, generator=torch.Generator().manual_seed(2)).to(dt).cuda()
    want = X.embed_backward(t, g, rows)
    whole = torch.full((rows + 2 * pad, 16), 7.0, dtype=dt, device="cuda")
    ws = X.Workspace.get(t.device, 0)
    ws[256:].fill_(old)  # (the header stays)
    X.test_set_sort_wait(16, True)
    try:
        X.embed_backward(t, g, rows, out=whole[pad:pad + rows, :dim])
    finally:
        X.test_set_sort_wait()
    with pytest.raises(X.LaplexError) as e:
        X.device_status()
    assert e.value.status == X.ETIMEOUT
    assert bool((whole[:pad] == 7).all()) and bool((whole[pad + rows:] == 7).all()) and bool((whole[:, dim:] == 7).all())
    X.device_status()  # cleared after being reported
    assert torch.equal(X.embed_backward(t, g, rows), want)
