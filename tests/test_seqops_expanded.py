"""Expanded tensors (strides of 0) are refused, by the binding or by the C call, as
the documentation says (no GPU needed)."""
import ctypes

import pytest
import torch

from exact_laplace_b200 import build
from exact_laplace_b200 import laplex as X

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    build.build()
    return X.lib()


def test_the_gradient_of_a_sum(L):
    with pytest.raises(X.LaplexError) as e:
        X._packed("dout", torch.ones(()).expand(6, 2, 8))
    assert e.value.status == X.EINVAL and "dout" in str(e.value) and "contiguous" in str(e.value)


@pytest.mark.parametrize("which", ["tokens", "heads"])
@pytest.mark.parametrize("at", range(4))
def test_rows_that_are_one(L, which, at):
    x = torch.zeros(6, 2, 8)
    x = x[:1].expand(6, 2, 8) if which == "tokens" else x[:, :1].expand(6, 2, 8)
    x = X._packed("x", x)  # its last dimension is contiguous: the C call looks at the strides
    rows = [ctypes.byref(X._Rows(256, 16, 8)) for _ in range(4)]
    rows[at] = ctypes.byref(X._Rows(256, x.stride(0), x.stride(1)))
    s = X._LinattnShape(6, 1, None, 2, 2, 8, 8, 256, 0.5, X.F32)
    q, k, v, o = rows
    assert L.laplex_linattn(ctypes.byref(s), q, k, v, None, o, None, P(256), 1 << 40, None) == X.EINVAL
    assert b"stride 0" in L.laplex_last_error()
