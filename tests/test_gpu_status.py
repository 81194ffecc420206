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
