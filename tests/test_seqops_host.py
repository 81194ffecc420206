"""Sequence operators: the C calls refuse bad arguments on the host, and the
binding refuses CPU tensors (no GPU needed)."""
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


def shape(tokens=100, seqs=2, cu=4096, hq=4, hkv=2, dk=64, dv=64, lam=256, dtype=3):
    return X._LinattnShape(tokens, seqs, cu, hq, hkv, dk, dv, lam, 0.5, dtype)


def rows(ptr=256, ts=256, hs=64):
    return ctypes.byref(X._Rows(ptr, ts, hs))


BIG = 1 << 40


def forward(L, s, q=None, k=None, v=None, o=None, state=None, ws=256, nb=BIG):
    r = rows()
    return L.laplex_linattn(ctypes.byref(s), q or r, k or r, v or r, P(state), o or r, None, P(ws), nb, None)


def refused(L, st, word):
    assert st == X.EINVAL, st
    assert word.encode() in L.laplex_last_error(), L.laplex_last_error()


@pytest.mark.parametrize("bad,word", [
    (dict(dtype=7), "dtype"), (dict(tokens=-1), "tokens"), (dict(tokens=1 << 31), "tokens"), (dict(hq=5), "hq"),
    (dict(hq=66, hkv=2), "hq"), (dict(hkv=0), "hkv"), (dict(dk=60), "dk"), (dict(dk=136), "dk"), (dict(dv=0), "dv"),
    (dict(seqs=-1), "seqs"), (dict(seqs=70000), "seqs"), (dict(seqs=0), "sequences"), (dict(cu=None, seqs=3), "divide"),
    (dict(cu=4097), "cu_seqlens"), (dict(lam=None), "log_decay"), (dict(lam=257), "log_decay")])
def test_shapes(L, bad, word):
    refused(L, forward(L, shape(**bad)), word)
    if word != "log_decay":
        n = ctypes.c_size_t()
        assert L.laplex_linattn_workspace_size(ctypes.byref(shape(**bad)), 0, ctypes.byref(n)) == X.EINVAL


@pytest.mark.parametrize("name", ["q", "k", "v", "o"])
def test_rows(L, name):
    for bad, word in ((rows(ptr=None), "NULL"), (rows(ptr=264), "aligned"), (rows(ts=32), "token stride"),
                      (rows(ts=260), "token stride"), (rows(hs=8), "head stride"), (rows(hs=68), "head stride"),
                      (rows(ts=0), "token stride"), (rows(ts=-256), "token stride")):
        st = forward(L, shape(), **{name: bad})
        refused(L, st, word)
        assert L.laplex_last_error().startswith(name.encode())
    assert L.laplex_linattn(ctypes.byref(shape()), *[None if name == n else rows() for n in ("q", "k", "v")], None,
                            None if name == "o" else rows(), None, P(256), BIG, None) == X.EINVAL


def test_rows_that_overlap(L):
    refused(L, forward(L, shape(), o=rows(ts=64, hs=64)), "overlap")


def test_states_and_workspaces(L):
    refused(L, forward(L, shape(), state=260), "state_in")
    refused(L, forward(L, shape(), ws=None), "workspace")
    refused(L, forward(L, shape(), ws=128), "workspace")
    s = shape(tokens=1 << 16)
    n = ctypes.c_size_t()
    sizes = []
    for call in (X.LINATTN_FORWARD, X.LINATTN_BACKWARD, X.LINATTN_BACKWARD_DECAY):
        assert L.laplex_linattn_workspace_size(ctypes.byref(s), call, ctypes.byref(n)) == X.OK
        sizes.append(n.value)
    assert 256 < sizes[0] <= sizes[1] <= sizes[2]
    assert forward(L, s, nb=sizes[0] - 1) == X.EWORKSPACE
    assert L.laplex_linattn_workspace_size(ctypes.byref(s), 3, ctypes.byref(n)) == X.EINVAL
    assert L.laplex_linattn_workspace_size(None, 0, ctypes.byref(n)) == X.EINVAL
    assert L.laplex_linattn_workspace_size(ctypes.byref(s), 0, None) == X.EINVAL
    st = L.laplex_linattn_backward(ctypes.byref(s), rows(), rows(), rows(), rows(), None, None, rows(), rows(), rows(),
                                   None, None, P(256), sizes[1] - 1, None)
    assert st == X.EWORKSPACE
    st = L.laplex_linattn_backward(ctypes.byref(s), rows(), rows(), rows(), rows(ptr=8), None, None, None, None, None,
                                   None, None, P(256), BIG, None)
    refused(L, st, "dout")
    st = L.laplex_linattn_backward(ctypes.byref(s), rows(), rows(), rows(), rows(), None, P(256), rows(), rows(), rows(),
                                   P(256), None, P(256), BIG, None)
    refused(L, st, "dstate_in")


def test_no_sequences_is_no_work(L):
    empty = rows(ptr=None)
    s = shape(tokens=0, seqs=0, cu=None)
    assert L.laplex_linattn(ctypes.byref(s), empty, empty, empty, None, empty, None, P(256), 256, None) == X.OK


def test_step(L):
    def call(s, states=256, slots=256, num=10, q=None):
        r = rows()
        return L.laplex_linattn_step(ctypes.byref(s), q or r, r, r, P(states), num, P(slots), r, None)

    refused(L, call(shape(tokens=4), states=None), "states")
    refused(L, call(shape(tokens=4), states=264), "states")
    refused(L, call(shape(tokens=4), num=-1), "num_slots")
    refused(L, call(shape(tokens=11), slots=None), "rows")
    refused(L, call(shape(tokens=4), slots=258), "slots")
    refused(L, call(shape(tokens=4, lam=None)), "log_decay")
    refused(L, call(shape(tokens=4), q=rows(ptr=24)), "q")


def test_embed(L):
    def look(table=256, ld=64, n_rows=10, dim=64, tok=256, tb=4, n=5, out=256, out_ld=64, dt=0):
        return L.laplex_embed(P(table), ld, n_rows, dim, P(tok), tb, n, 1.0, P(out), out_ld, dt, None)

    for bad, word in ((dict(table=None), "table"), (dict(table=8), "table"), (dict(ld=63), "table"), (dict(dim=0), "dim"),
                      (dict(tok=None), "tokens"), (dict(tok=258), "tokens"), (dict(tb=2), "token_bytes"),
                      (dict(n=-1), "n ="), (dict(n=1 << 31), "n ="), (dict(out=None), "out"), (dict(out_ld=3), "out"),
                      (dict(dt=4), "dtype"), (dict(n_rows=-1), "rows")):
        refused(L, look(**bad), word)

    def grad(tok=256, tb=4, n=5, g=256, g_ld=64, n_rows=10, dim=64, out=256, ld=64, dt=3, odt=3, ws=256, nb=BIG):
        return L.laplex_embed_backward(P(tok), tb, n, P(g), g_ld, n_rows, dim, 1.0, 0, P(out), ld, dt, odt, P(ws), nb, None)

    for bad, word in ((dict(g=None), "g is"), (dict(g_ld=60), "g:"), (dict(out=None), "dtable"), (dict(ld=60), "dtable"),
                      (dict(odt=2), "out_dtype"), (dict(odt=1), "out_dtype"), (dict(dt=1, odt=0), "out_dtype"),
                      (dict(ws=None), "workspace"), (dict(ws=16), "workspace"), (dict(tb=1), "token_bytes")):
        refused(L, grad(**bad), word)
    n = ctypes.c_size_t()
    assert L.laplex_embed_backward_workspace_size(1000, 100, 64, 3, ctypes.byref(n)) == X.OK
    assert grad(n=1000, n_rows=100, nb=n.value - 1) == X.EWORKSPACE
    assert L.laplex_embed_backward_workspace_size(1000, 100, 64, 3, None) == X.EINVAL


def test_other_calls_refuse_the_16_bit_types(L):
    for dt in (X.F16, X.BF16):
        st = L.laplex_matvec_sym(P(256), None, 10, P(256), P(512), 1, dt, P(256), 1 << 20, None)
        refused(L, st, "dtype")


def test_binding_refuses(L):
    x = torch.zeros(4, 2, 8)
    lam = torch.zeros(2)
    for call in (lambda: X.linattn(x, x, x, lam), lambda: X.linattn_backward(x, x, x, lam, x),
                 lambda: X.linattn_step(x, x, x, lam, torch.zeros(4, 2, 8, 8)),
                 lambda: X.embed(torch.zeros(3, 8), torch.zeros(2, dtype=torch.int32)),
                 lambda: X.embed_backward(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 8), 3)):
        with pytest.raises(X.LaplexError) as e:
            call()
        assert e.value.status == X.EINVAL and "CUDA" in str(e.value)
    with pytest.raises(X.LaplexError):
        X._packed("q", torch.zeros(4, 2, 16)[..., ::2])
    with pytest.raises(X.LaplexError):
        X._packed("q", torch.zeros(4, 8))
    with pytest.raises(X.LaplexError):
        X._packed("q", torch.zeros(6, 5, 2, 8)[::2])
    with pytest.raises(X.LaplexError):
        X._seq_dt(x, x.half())
    with pytest.raises(X.LaplexError):
        X._seq_dt(x.int())
    with pytest.raises(X.LaplexError):
        X._shape(x, x[:3], x, 1, None, lam, None, X.F32)
    with pytest.raises(X.LaplexError):
        X._shape(x, x, x, 1, None, lam.double(), None, X.F32)
    with pytest.raises(X.LaplexError):
        X._seqs(x, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(X.LaplexError):
        X._tokens(torch.zeros(3))
