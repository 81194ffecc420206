"""Decayed linear attention over many chunks of the largest heads: launches that
fill the GPU, cut and uncut sequences, and bounds that see a lost or a misplaced
term (the worst-case bounds beside the shapes' tests grow with the sums of
magnitudes, which cancel in a long sequence).

Exact: with lam = 0, scale = 1 and small whole numbers every product, weight and
state is a whole number that the 16-bit types hold, so an output is the
definition's, rounded once.

Rms: roundings are independent, at most u = eps / 2 of what they round and so u /
sqrt(3) of it in the mean square.  An output of independent terms takes one
rounding of its terms (a weight, or the state's entry) and its own: sqrt(2 / 3) u
of the outputs' rms, and 1e-4 for the fp32 part as in the other bounds.
"""
import functools

import numpy as np
import pytest
import torch

from exact_laplace_b200 import laplex as X
from oracle import seq
from test_gpu_linattn import DT, Case, np64, tol_acc

pytestmark = pytest.mark.gpu

HEADS = [(2, 2, 128, 128), (8, 2, 128, 128), (2, 2, 64, 64), (3, 1, 72, 128), (2, 2, 128, 40)]
LENS = [(2500,), (700, 0, 1900, 3, 129), (1024, 1024), (300,)]


def whole_numbers(c, seed):
    """q, k, v, do of -1, 0, 1 (mostly 0), states of -3 to 3; scale = 1."""
    g = torch.Generator().manual_seed(seed)

    def few(x):
        z = torch.randint(-1, 2, x.shape, generator=g) * (torch.rand(x.shape, generator=g) < 0.2)
        return z.to(x.dtype).cuda()

    c.q, c.k, c.v, c.do = (few(x) for x in (c.q, c.k, c.v, c.do))
    if c.s0 is not None:
        c.s0, c.ds = (torch.randint(-3, 4, x.shape, generator=g).to(x.dtype).cuda() for x in (c.s0, c.ds))
    c.scale = 1.0


def held(*xs):
    """Whether the 16-bit types hold these whole numbers, and so everything in between (bf16: up to 256)."""
    return all(np.max(np.abs(x), initial=0.0) <= 256 for x in xs)


def same(y, ref, dt, what):
    want = torch.from_numpy(ref).to(y.dtype).cuda()
    assert torch.equal(y, want), f"{what}: {int((y != want).sum())} of {y.numel()} differ"


@functools.lru_cache(maxsize=2)
def exact_of(lens, heads, state, seed):
    c = Case("fp32", lens, *heads, state=state, lam=[0.0] * heads[1])
    whole_numbers(c, seed)
    q, k, v, do, s0, ds = c.host()
    lam = np64(c.lam)
    ro, rend = seq.linattn(q, k, v, lam, 1.0, lens, s0)
    r = seq.linattn_backward(q, k, v, lam, do, 1.0, lens, s0, ds)
    assert held(rend, r["dstate"])
    return ro, rend, r


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_whole_numbers(dt, heads, lens, state):
    c = Case(dt, lens, *heads, state=state, lam=[0.0] * heads[1])
    whole_numbers(c, len(lens))
    ro, rend, r = exact_of(lens, heads, state, len(lens))
    o, end = c.run_forward()
    same(o, ro, dt, "o")
    same(end, rend, dt, "state")
    g = c.run_backward(return_dstate=True, return_dlog_decay=True)
    for name in ("dq", "dk", "dv", "dstate"):
        same(getattr(g, name), r[name], dt, name)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("state", [False, True])
def test_whole_numbers_of_many_sequences(dt, state):
    """More blocks than the GPU has SMs, sequences of a known length, none cut."""
    n, length = 40, 400
    c = Case(dt, (length,) * n, 8, 8, 128, 128, state=state, lam=[0.0] * 8)
    whole_numbers(c, 7)
    four = [x.contiguous().view(n, length, *x.shape[1:]) for x in (c.q, c.k, c.v, c.do)]
    ro, rend, r = exact_of((length,) * n, (8, 8, 128, 128), state, 7)
    o, end = X.linattn(*four[:3], c.lam, scale=1.0, state=c.s0, return_state=True)
    same(o.flatten(0, 1), ro, dt, "o")
    same(end, rend, dt, "state")
    g = X.linattn_backward(*four[:3], c.lam, four[3], scale=1.0, state=c.s0, dstate=c.ds, return_dstate=True)
    for name in ("dq", "dk", "dv"):
        same(getattr(g, name).flatten(0, 1), r[name], dt, name)
    same(g.dstate, r["dstate"], dt, "dstate")


def rms(y, ref, what, dt, heads_at=1):
    """Per head: the error's rms against the outputs'."""
    u = torch.finfo(DT[dt]).eps / 2
    bound = (2 / 3) ** 0.5 * u + 1e-4
    e = np64(y) - ref
    for h in range(ref.shape[heads_at]):
        a, b = np.take(e, h, heads_at), np.take(ref, h, heads_at)
        err = np.sqrt(np.mean(a ** 2)) / np.sqrt(np.mean(b ** 2))
        assert err <= bound, f"{what}, head {h}: rms error {err:.3e} > {bound:.3e}"


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("heads", HEADS[:3], ids=str)
@pytest.mark.parametrize("lens", [(2500,), (700, 1900)], ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_rms(dt, heads, lens, state):
    c = Case(dt, lens, *heads, state=state, lam=[-0.002, -0.05][:heads[1]], seed=3)
    if state:  # of the size that the tokens' own states have
        c.s0, c.ds = 4 * c.s0, c.ds
    (ro, rend), (_, nend) = c.forward_ref()
    o, end = c.run_forward()
    rms(o, ro, "o", dt)
    assert np.max(np.abs(np64(end) - rend) / nend) <= tol_acc(dt)
    r, _ = c.backward_ref()
    g = c.run_backward()
    for name in ("dq", "dk", "dv"):
        rms(getattr(g, name), r[name], name, dt)
