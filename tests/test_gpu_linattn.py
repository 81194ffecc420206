"""Decayed linear attention on the GPU against its fp64 definition: prompts,
gradients and single tokens, in the four types.

Tolerances, as normalised errors max |y - y_ref| / N with N the same sum over
absolute values (scale sum e^{lam (t - s)} |q||k||v|, ...): fp64 1e-10 and fp32
1e-4 as for the library's other products.  16-bit rows: every term of an output
takes at most one rounding to the rows' type before the sum (its weight, or the
state's entry) and the output one more, each at most u = eps / 2 of the term, so
(1 + u)^2 - 1 plus the fp32 part, 1e-4.  States and the decay's gradient are
not rounded to 16 bits: 1e-4.  fp16 weights and states are scaled by a power of
two before their rounding, whose absolute part is 2^-25 of the largest of the
row (of the state): `floor` allows that against the row's largest weight.
"""
import numpy as np
import pytest
import torch

from exact_laplace_b200 import laplex as X
from oracle import seq

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp64": torch.float64}
ALL = list(DT)
DECAYS = [-0.5, -0.01, -0.07, -1e-3, -3.0, -0.2]


def tol_rows(dt):
    u = torch.finfo(DT[dt]).eps / 2
    return {"fp64": 1e-10, "fp32": 1e-4}.get(dt, (1 + u) ** 2 - 1 + 1e-4)


def tol_acc(dt):
    return 1e-10 if dt == "fp64" else 1e-4


def acc(dt):
    return torch.float64 if dt == "fp64" else torch.float32


def np64(t):
    return t.detach().cpu().double().numpy()


def check(y, ref, norm, tol, what, floor=0.0):
    y = np64(y)
    assert np.all(np.isfinite(y)), f"{what}: not finite"
    err = np.max((np.abs(y - ref) - floor) / np.where(norm > 0, norm, 1.0)) if y.size else 0.0
    assert err <= tol, f"{what}: normalised error {err:.3e} > {tol:.3e}"


class Case:
    """Inputs of one call, their exact results and their normalisers."""

    def __init__(self, dt, lens, hq=2, hkv=1, dk=64, dv=64, state=True, lam=None, seed=0, tail=0, sliced=False):
        rng = np.random.default_rng(seed + 1000 * sum(lens) + hq)
        self.dt, self.lens, self.n = dt, lens, len(lens)
        t = sum(lens) + tail
        self.shape = (t, hq, hkv, dk, dv)

        def normal(*shape):
            return torch.from_numpy(rng.standard_normal(shape)).to(DT[dt]).cuda()

        if sliced:
            row = normal(t, (hq + hkv) * dk + hkv * dv + 16)
            q, k, v, _ = row.split([hq * dk, hkv * dk, hkv * dv, 16], 1)
            self.q, self.k, self.v = q.unflatten(1, (hq, dk)), k.unflatten(1, (hkv, dk)), v.unflatten(1, (hkv, dv))
        else:
            self.q, self.k, self.v = normal(t, hq, dk), normal(t, hkv, dk), normal(t, hkv, dv)
        self.do = normal(t, hq, dv)
        lam = DECAYS[:hkv] if lam is None else lam
        self.lam = torch.tensor(lam, dtype=acc(dt)).cuda()
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
        big = lambda: torch.from_numpy(3 * rng.standard_normal((self.n, hkv, dk, dv))).to(acc(dt)).cuda()
        self.s0, self.ds = (big(), big()) if state else (None, None)
        self.scale = dk ** -0.5

    def host(self, absolute=False):
        f = (lambda x: None if x is None else np.abs(np64(x))) if absolute else (lambda x: None if x is None else np64(x))
        return [f(x) for x in (self.q, self.k, self.v, self.do, self.s0, self.ds)]

    def forward_ref(self):
        lam = np64(self.lam)
        q, k, v, _, s0, _ = self.host()
        a = self.host(True)
        return (seq.linattn(q, k, v, lam, self.scale, self.lens, s0),
                seq.linattn(a[0], a[1], a[2], lam, abs(self.scale), self.lens, a[4]))

    def backward_ref(self):
        lam = np64(self.lam)
        q, k, v, do, s0, ds = self.host()
        a = self.host(True)
        return (seq.linattn_backward(q, k, v, lam, do, self.scale, self.lens, s0, ds),
                seq.linattn_backward(a[0], a[1], a[2], lam, a[3], abs(self.scale), self.lens, a[4], a[5]))

    def used(self):
        return slice(0, sum(self.lens))

    def run_forward(self, **kw):
        return X.linattn(self.q, self.k, self.v, self.lam, scale=self.scale, cu_seqlens=self.cu, state=self.s0,
                         return_state=True, **kw)

    def run_backward(self, **kw):
        return X.linattn_backward(self.q, self.k, self.v, self.lam, self.do, scale=self.scale, cu_seqlens=self.cu,
                                  state=self.s0, dstate=self.ds, **kw)

    def check_forward(self, o, end):
        (ro, rend), (no, nend) = self.forward_ref()
        u = self.used()
        # (fp16) weights and states are rounded on a grid relative to their largest
        floor = 2.0 ** -24 * np.max(no, initial=0.0) if self.dt == "fp16" else 0.0
        check(o[u], ro[u], no[u], tol_rows(self.dt), "o", floor)
        check(end, rend, nend, tol_acc(self.dt), "state")

    def check_backward(self, g):
        r, n = self.backward_ref()
        u = self.used()
        for name in ("dq", "dk", "dv"):
            floor = 2.0 ** -24 * np.max(n[name], initial=0.0) if self.dt == "fp16" else 0.0
            check(getattr(g, name)[u], r[name][u], n[name][u], tol_rows(self.dt), name, floor)
        if g.dstate is not None:
            check(g.dstate, r["dstate"], n["dstate"], tol_acc(self.dt), "dstate")
        if g.dlog_decay is not None:
            check(g.dlog_decay, r["dlam"], n["dlam"], tol_acc(self.dt), "dlog_decay")


LENGTHS = [[1], [2], [16], [127], [128], [129], [255, 1, 0, 64, 200], [0, 0, 5]]
SHAPES = [(1, 1, 8, 8), (4, 2, 64, 64), (3, 1, 72, 104), (2, 2, 128, 128), (5, 5, 128, 40), (2, 1, 24, 128)]


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_forward_lengths(dt, lens):
    c = Case(dt, lens)
    c.check_forward(*c.run_forward())


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_forward_shapes(dt, shape, state):
    c = Case(dt, [130, 61], *shape, state=state, sliced=True)
    c.check_forward(*c.run_forward())


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("lens", [[2500], [700, 1900, 3]], ids=str)
def test_forward_cut_into_segments(dt, lens):
    c = Case(dt, lens, 2, 2, 64, 128, lam=[-0.002, -0.3])
    c.check_forward(*c.run_forward())


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_backward_lengths(dt, lens):
    c = Case(dt, lens)
    c.check_backward(c.run_backward(return_dlog_decay=True))


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_backward_shapes(dt, shape, state):
    c = Case(dt, [130, 61], *shape, state=state, sliced=True)
    g = c.run_backward(return_dstate=True, return_dlog_decay=True)
    c.check_backward(g)


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("lens", [[2500], [700, 1900, 3]], ids=str)
def test_backward_cut_into_segments(dt, lens):
    c = Case(dt, lens, 4, 2, 64, 128, lam=[-0.002, -0.3])
    c.check_backward(c.run_backward(return_dlog_decay=True))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lam", [0.0, -20.0, -1e4, float("-inf")])
def test_decays_at_the_ends(dt, lam):
    c = Case(dt, [200, 30], 2, 2, 64, 64, lam=[lam, -0.1])
    with np.errstate(over="ignore"):
        c.check_forward(*c.run_forward())
        c.check_backward(c.run_backward())


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_large_values(dt):
    """Products past the 16-bit types' largest values inside the sums: the output
    is representable, the weights and states are not (fp16: 65504)."""
    c = Case(dt, [300], 1, 1, 64, 64, lam=[-0.001])
    c.q *= 64
    c.k *= 64
    c.v *= 16
    c.s0 *= 1e5
    c.scale = 2.0 ** -14
    c.check_forward(*c.run_forward())


@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [[0], [5], [40, 41, 90], [127, 128], [299]], ids=str)
def test_no_token_reaches_an_earlier_output(dt, which, bad, at):
    """NaN and Inf in a row of k or v: the earlier rows of o keep their values,
    the later ones take it over in the columns it reaches."""
    c = Case(dt, [300, 50], 2, 1, 64, 64)
    (ro, _), (no, _) = c.forward_ref()
    x = getattr(c, which)
    for t in at:
        x[t, 0, 3] = bad
    o, _ = c.run_forward()
    first = min(at)
    check(o[:first], ro[:first], no[:first], tol_rows(dt), "rows before")
    check(o[300:], ro[300:], no[300:], tol_rows(dt), "the next sequence")
    if which == "v":
        assert not torch.isfinite(o[first:300, :, 3]).any()
        rest = [j for j in range(64) if j != 3]
        check(o[first:300, :, rest], ro[first:300][:, :, rest], no[first:300][:, :, rest], tol_rows(dt), "other columns")
    else:
        assert not torch.isfinite(o[first]).any()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_nan_stays_with_its_sequence_in_the_gradients(dt):
    c = Case(dt, [70, 60, 30], 2, 1, 64, 64)
    r, n = c.backward_ref()
    for x in (c.q, c.k, c.v, c.do):
        x[75:80] = float("nan")
    g = c.run_backward()
    for name in ("dq", "dk", "dv"):
        for sl in (slice(0, 70), slice(130, 160)):
            check(getattr(g, name)[sl], r[name][sl], n[name][sl], tol_rows(dt), name)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rows_behind_the_last_sequence_stay(dt):
    c = Case(dt, [100, 33], 2, 1, 64, 64, tail=50)
    for x in (c.q, c.k, c.v, c.do):
        x[133:] = float("nan")
    o = torch.full((183, 2, 64), 7.0, dtype=DT[dt], device="cuda")
    _, end = c.run_forward(out=o)
    assert torch.all(o[133:] == 7)
    for x in (c.q, c.k, c.v, c.do):
        x[133:] = 0
    c.check_forward(o, end)
    outs = tuple(torch.full_like(x, 5.0).contiguous() for x in (c.q, c.k, c.v))
    g = c.run_backward(out=outs)
    assert all(torch.all(x[133:] == 5) for x in outs)
    c.check_backward(g)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_equal_lengths_four_dimensions_and_head_major_rows(dt):
    c = Case(dt, [150] * 3, 4, 2, 64, 64)
    want, _ = c.run_forward()
    four = [x.contiguous().view(3, 150, *x.shape[1:]) for x in (c.q, c.k, c.v)]
    o, end = X.linattn(*four, c.lam, scale=c.scale, state=c.s0, return_state=True)
    assert o.shape == (3, 150, 4, 64)
    # (known and unknown lengths may be cut differently, and so round differently: the same bounds, not the same bits)
    c.check_forward(o.view_as(want), end)
    again, _ = X.linattn(*four, c.lam, scale=c.scale, state=c.s0, return_state=True)
    assert torch.equal(again, o)
    major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c.q, c.k, c.v)]
    o, _ = X.linattn(*major, c.lam, scale=c.scale, cu_seqlens=c.cu, state=c.s0, return_state=True)
    assert torch.equal(o, want)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[90], [3000]], ids=str)
def test_state_in_place_and_prompts_in_pieces(dt, lens):
    """A prompt in two calls through its state, written over the one read."""
    c = Case(dt, lens, 2, 1, 64, 64)
    state = c.s0.clone()
    cut = lens[0] // 3
    for sl in (slice(0, cut), slice(cut, None)):
        o, got = X.linattn(c.q[sl], c.k[sl], c.v[sl], c.lam, scale=c.scale, state=state, state_out=state)
        assert got is state
    (ro, rend), (no, nend) = c.forward_ref()
    check(o, ro[cut:], no[cut:], tol_rows(dt), "o")
    check(state, rend, nend, 2 * tol_acc(dt), "state")  # two calls


def test_same_bits_on_every_run():
    for lens in ([600, 5], [4000]):
        c = Case("bf16", lens, 4, 2, 64, 128)
        a, b = c.run_forward(), c.run_forward()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        a, b = c.run_backward(return_dlog_decay=True), c.run_backward(return_dlog_decay=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_gradients_that_are_not_asked_for(dt):
    """The C call leaves out what is NULL and computes the rest.  (16-bit rows: not
    to the last bit as beside the others, since K's weights take a third part only
    where a state leaves the call; the bounds against the definition are the same.)"""
    import ctypes
    c = Case(dt, [300, 20], 4, 2, 64, 64)
    g = c.run_backward()
    s, _ = X._shape(c.q, c.k, c.v, 2, c.cu, c.lam, c.scale, X._seq_dt(c.q))
    r, n = c.backward_ref()
    for keep in ("dq", "dk", "dv", "dstate"):
        new = {n: torch.empty_like(getattr(g, n)) if n == keep else None for n in ("dq", "dk", "dv", "dstate")}
        ws = X._linattn_ws(s, X.LINATTN_BACKWARD, c.q.device, X._raw_stream(c.q.device))
        X._check(X.lib().laplex_linattn_backward(
            ctypes.byref(s), X._rows(c.q), X._rows(c.k), X._rows(c.v), X._rows(c.do), X._ptr(c.s0), X._ptr(c.ds),
            X._rows(new["dq"]), X._rows(new["dk"]), X._rows(new["dv"]), X._ptr(new["dstate"]), None, X._ptr(ws),
            ws.numel(), X._stream(c.q.device)))
        check(new[keep], r[keep], n[keep], tol_acc(dt) if keep == "dstate" else tol_rows(dt), keep)
        if dt == "fp32":
            assert torch.equal(new[keep], getattr(g, keep)), keep


# ----------------------------------------------------------------------------- single tokens

@pytest.mark.parametrize("dt", ALL)
@pytest.mark.parametrize("shape", SHAPES + [(32, 1, 64, 64), (7, 1, 128, 128)], ids=str)
@pytest.mark.parametrize("rows", [1, 3, 160])
def test_step(dt, shape, rows):
    hq, hkv, dk, dv = shape
    c = Case(dt, [1] * rows, hq, hkv, dk, dv, sliced=True)
    states = torch.zeros((rows + 5, hkv, dk, dv), dtype=acc(dt), device="cuda")
    slots = torch.randperm(rows + 5, generator=torch.Generator().manual_seed(rows))[:rows].int().cuda()
    states[slots.long()] = c.s0
    untouched = states.clone()
    o = X.linattn_step(c.q, c.k, c.v, c.lam, states, slots=slots, scale=c.scale)
    c.check_forward(o, states[slots.long()])
    rest = [i for i in range(rows + 5) if i not in set(slots.tolist())]
    assert torch.equal(states[rest], untouched[rest])
    again = c.s0.clone()
    assert torch.equal(X.linattn_step(c.q, c.k, c.v, c.lam, again, scale=c.scale), o)
    assert torch.equal(again, states[slots.long()])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_step_rows_of_one_slot_and_of_none(dt):
    """Rows of one slot are applied in row order: the prompt of those rows."""
    c = Case(dt, [6], 4, 2, 64, 128)
    states = torch.zeros((4, 2, 64, 128), dtype=acc(dt), device="cuda")
    states[2] = c.s0[0]
    other = torch.randn_like(states[1])
    states[1] = other
    x = lambda t: torch.cat([t[:2], t[:1], t[2:5], t[:1], t[5:]])
    slots = torch.tensor([2, 2, -1, 2, 2, 2, 4, 2], dtype=torch.int32, device="cuda")
    o = X.linattn_step(x(c.q), x(c.k), x(c.v), c.lam, states, slots=slots, scale=c.scale)
    assert torch.all(o[[2, 6]] == 0)
    c.check_forward(o[[0, 1, 3, 4, 5, 7]], states[2:3])
    assert torch.equal(states[1], other) and torch.all(states[[0, 3]] == 0)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_step_many_tokens_of_a_slow_decay(dt):
    """2000 single tokens against one prompt: the decays' roundings do not add up."""
    n = 2000
    c = Case(dt, [n], 1, 1, 16, 16, lam=[-1e-3])
    states = c.s0.clone()
    o = torch.empty((n, 1, 16), dtype=DT[dt], device="cuda")
    for t in range(n):
        X.linattn_step(c.q[t:t + 1], c.k[t:t + 1], c.v[t:t + 1], c.lam, states, scale=c.scale, out=o[t:t + 1])
    (ro, rend), (no, nend) = c.forward_ref()
    check(states, rend, nend, 1e-5, "state")
    check(o, ro, no, tol_rows(dt), "o")
    _, end = c.run_forward()
    check(end, rend, nend, 1e-5, "the prompt's state")


# ----------------------------------------------------------------------------- streams, graphs, together

def test_other_stream_and_two_graphs():
    cs = [Case("bf16", [700, 30], 2, 1, 64, 64), Case("bf16", [2600], 2, 1, 64, 64, seed=4)]
    eager = [(c.run_forward(), c.run_backward(return_dlog_decay=True)) for c in cs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = [(c.run_forward(), c.run_backward(return_dlog_decay=True)) for c in cs]
    torch.cuda.synchronize()
    for (f, b), (f2, b2) in zip(eager, other):
        assert all(torch.equal(x, y) for x, y in zip(f + b, f2 + b2))
    graphs = []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = (c.run_forward(), c.run_backward(return_dlog_decay=True))
        graphs.append((g, res))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for st, (g, _) in zip((a, b), graphs):  # at the same time
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (f, b2), (_, (f2, b3)) in zip(eager, graphs):
            assert all(torch.equal(x, y) for x, y in zip(f + b2, f2 + b3))
    # other data in the same buffers
    c, (g, res) = cs[0], graphs[0]
    c.q.normal_()
    c.v.normal_()
    g.replay()
    torch.cuda.synchronize()
    f, b = c.run_forward(), c.run_backward(return_dlog_decay=True)
    assert all(torch.equal(x, y) for x, y in zip(f + b, res[0] + res[1]))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_tokens_to_gradients(dt):
    """A padded batch through the operators as a model's first layer uses them:
    embed, linattn, a loss, their gradients down to the table's; then the same
    sequence continued token by token."""
    rng = np.random.default_rng(3)
    h, d, rows = 2, 64, 50
    tok = torch.from_numpy(rng.integers(0, rows, (3, 70))).cuda()
    tok[1, 40:] = -1
    table = torch.from_numpy(rng.standard_normal((rows, h * d))).to(DT[dt]).cuda()
    lam = torch.tensor([-0.1, -0.01], device="cuda")
    x = X.embed(table, tok, scale=0.5)
    q = x.view(3, 70, h, d)
    o, end = X.linattn(q, q, q, lam, return_state=True)
    g = X.linattn_backward(q, q, q, lam, torch.ones_like(o))
    dx = (g.dq.float() + g.dk.float() + g.dv.float()).to(DT[dt])
    dt_ = X.embed_backward(tok, dx.view(3, 70, h * d), rows, scale=0.5, dtype=torch.float32)

    xr = seq.embed(np64(table), tok.flatten().cpu().numpy(), 0.5)
    # the rounded rows are what the attention reads
    xq = np64(x).reshape(210, h, d)
    assert np.max(np.abs(np64(x).reshape(210, -1) - xr)) <= torch.finfo(DT[dt]).eps / 2 * np.max(np.abs(xr))
    r = seq.linattn_backward(xq, xq, xq, np64(lam), np.ones((210, h, d)), d ** -0.5, [70] * 3)
    n = seq.linattn_backward(abs(xq), abs(xq), abs(xq), np64(lam), np.ones((210, h, d)), d ** -0.5, [70] * 3)
    want = seq.embed_backward(tok.flatten().cpu().numpy(), (r["dq"] + r["dk"] + r["dv"]).reshape(210, -1), rows, 0.5)
    norm = seq.embed_backward(tok.flatten().cpu().numpy(), (n["dq"] + n["dk"] + n["dv"]).reshape(210, -1), rows, 0.5)
    u = torch.finfo(DT[dt]).eps / 2
    check(dt_, want, norm, tol_rows(dt) * (1 + u) + u + 1e-4, "the table's gradient")  # dx is rounded once more
    # two more tokens of sequences 0 and 2
    new = torch.tensor([7, 9, 11, 13], device="cuda")
    xn = X.embed(table, new, scale=0.5).view(4, h, d)
    slots = torch.tensor([0, 2, 0, 2], dtype=torch.int32, device="cuda")
    on = X.linattn_step(xn, xn, xn, lam, end, slots=slots)
    for s, at in ((0, [0, 2]), (2, [1, 3])):
        full = np.concatenate([xq[70 * s:70 * s + 70], np64(xn[at])])
        ro, _ = seq.linattn(full, full, full, np64(lam), d ** -0.5, [72])
        no, _ = seq.linattn(abs(full), abs(full), abs(full), np64(lam), d ** -0.5, [72])
        check(on[at], ro[70:], no[70:], tol_rows(dt), "continued")


# ----------------------------------------------------------------------------- calls at the edges

@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hq,hkv", [(32, 1), (24, 2), (34, 2)])
def test_large_groups(dt, hq, hkv):
    c = Case(dt, [150, 61], hq, hkv, 64, 32)
    c.check_forward(*c.run_forward())
    c.check_backward(c.run_backward(return_dlog_decay=True))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_states_that_grow(dt):
    # e^{0.01 * 400} = 55: a positive log decay is a growth
    c = Case(dt, [400, 33], 2, 2, 64, 64, lam=[0.01, 0.002])
    c.check_forward(*c.run_forward())
    c.check_backward(c.run_backward())


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scale", [0.0, -2.0, 1e-6])
def test_scales(dt, scale):
    c = Case(dt, [300, 20], 2, 1, 64, 72, state=False)
    c.scale = scale
    if dt == "fp16" and scale == 1e-6:  # outputs in fp16's subnormal range: rounded on its grid of 2^-24
        o, _ = c.run_forward()
        (ro, _), (no, _) = c.forward_ref()
        assert np.max(np.abs(np64(o) - ro) - tol_rows(dt) * no) <= 2.0 ** -24
        return
    c.check_forward(*c.run_forward())
    c.check_backward(c.run_backward())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_many_sequences(dt):
    lens = [0] * 65535
    for i in range(0, len(lens), 7):
        lens[i] = i % 3 + 1
    c = Case(dt, lens, 1, 1, 8, 8, state=False)
    c.check_forward(*c.run_forward())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_many_heads(dt):
    c = Case(dt, [40, 9], 300, 300, 16, 8, lam=[-0.01 * (i % 40) for i in range(300)])
    c.check_forward(*c.run_forward())
    c.check_backward(c.run_backward(return_dlog_decay=True))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32", "fp64"])
def test_no_tokens(dt):
    c = Case(dt, [0, 0, 0], 2, 1, 64, 64)
    o, end = c.run_forward()
    assert o.shape == (0, 2, 64) and torch.equal(end, c.s0)
    g = c.run_backward(return_dlog_decay=True)
    # no token: the state goes through as it came (e^lam R_0 with R_0 = e^-lam dstate)
    assert torch.equal(g.dstate, c.ds)
    assert torch.equal(g.dlog_decay, torch.zeros_like(g.dlog_decay))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_offsets_past_32_bits(dt):
    # rows 2^28 elements apart: the tenth starts past 2^31 elements
    ts, n = (1 << 28) + 64, 10
    c = Case(dt, [n], 1, 1, 64, 64)
    if torch.cuda.mem_get_info()[0] < 3 * n * ts * c.q.element_size():
        pytest.skip("not enough memory")
    far = []
    for x in (c.q, c.k):
        buf = torch.empty(n * ts, dtype=x.dtype, device="cuda")
        y = buf.as_strided((n, 1, 64), (ts, 64, 1))
        y.copy_(x)
        far.append(y)
    c.q, c.k = far
    c.check_forward(*c.run_forward())
    c.check_backward(c.run_backward())
    one = slice(n - 1, n)
    states = c.s0.clone()
    o = X.linattn_step(c.q[one], c.k[one], c.v[one], c.lam, states, scale=c.scale)
    ro, _ = seq.linattn(np64(c.q)[one], np64(c.k)[one], np64(c.v)[one], np64(c.lam), c.scale, [1], np64(c.s0))
    no, _ = seq.linattn(abs(np64(c.q)[one]), abs(np64(c.k)[one]), abs(np64(c.v)[one]), np64(c.lam), c.scale, [1],
                        abs(np64(c.s0)))
    check(o, ro, no, tol_rows(dt), "step")


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_graph_replayed_with_other_lengths(dt):
    """Lengths are read on the device: a captured call serves every packing of its
    tokens, cut into segments or not."""
    lens = [[1500, 200, 0, 1300], [0, 3000, 0, 0], [1, 999, 1000, 1000], [40, 50, 60, 70]]
    c = Case(dt, lens[0], 2, 1, 64, 64)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run_forward(), c.run_backward()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        res = (c.run_forward(), c.run_backward(return_dlog_decay=True))
    for x in lens:
        c.lens = x
        c.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32))
        for t in (c.q, c.k, c.v, c.do):
            t.normal_()
        g.replay()
        torch.cuda.synchronize()
        c.check_forward(*res[0])
        c.check_backward(res[1])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("bounds", [[0, 900, 300, 700], [5, -7, 2000, 640], [700, 700, 0, 700], [0, 2 ** 31 - 1, -2 ** 31, 9]],
                         ids=str)
def test_bounds_that_do_not_ascend_stay_inside(dt, bounds):
    """Unspecified results, but nothing outside the tensors is written, and the
    device stays usable."""
    t, pad = 700, 64
    c = Case(dt, [300, 300, 100], 2, 1, 64, 64)
    c.cu = torch.tensor(bounds, dtype=torch.int32).cuda()
    whole = torch.full((t + 2 * pad, 2, 64), 7.0, dtype=DT[dt], device="cuda")
    out = whole[pad:pad + t]
    X.linattn(c.q, c.k, c.v, c.lam, cu_seqlens=c.cu, state=c.s0, return_state=True, out=out)
    c.run_backward(return_dlog_decay=True)
    torch.cuda.synchronize()
    assert bool((whole[:pad] == 7).all()) and bool((whole[pad + t:] == 7).all())
    X.device_status()
    d = Case(dt, [300, 300, 100], 2, 1, 64, 64)
    d.check_forward(*d.run_forward())


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_nan_decay_stays_in_its_head(dt):
    c = Case(dt, [200], 2, 2, 64, 64, lam=[-0.1, float("nan")])
    o, end = c.run_forward()
    d = Case(dt, [200], 2, 2, 64, 64, lam=[-0.1, -0.1])
    o2, end2 = d.run_forward()
    assert torch.equal(o[:, 0], o2[:, 0]) and torch.equal(end[:, 0], end2[:, 0])
    assert bool(torch.isnan(end[:, 1]).all())


@pytest.mark.parametrize("dt", ["bf16", "fp64"])
def test_differences(dt):
    """The gradients against central differences of the fp64 forward call on the
    same values, along one direction of each input, over several segments."""
    c = Case(dt, [1200, 40], 2, 1, 16, 24)
    w = Case("fp64", [1200, 40], 2, 1, 16, 24)
    w.q, w.k, w.v, w.do = (x.double() for x in (c.q, c.k, c.v, c.do))
    w.lam, w.s0, w.ds = c.lam.double(), c.s0.double(), c.ds.double()
    g = c.run_backward(return_dlog_decay=True)

    def loss():
        o, end = w.run_forward()
        return float((o * w.do).sum() + (end * w.ds).sum())

    _, n = w.backward_ref()
    for x, grad, name in ((w.q, g.dq, "dq"), (w.k, g.dk, "dk"), (w.v, g.dv, "dv"), (w.s0, g.dstate, "dstate"),
                          (w.lam, g.dlog_decay, "dlam")):
        step = torch.randn(x.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(5)).cuda()
        h = 1e-4 if name == "dlam" else 1e-2
        keep = x.clone()
        x.copy_(keep + h * step)
        up = loss()
        x.copy_(keep - h * step)
        down = loss()
        x.copy_(keep)
        mine = float((grad.double() * step).sum())
        size = float((torch.from_numpy(n[name]).cuda() * step.abs()).sum())
        # The loss is linear in all but lam: the difference is exact up to fp64's rounding.  In lam it is off by
        # (h step)^2 / 6 of the third derivative, whose terms are d^2 times the first's: with e^{-d / 2}
        # sum d^3 / sum d = 24, so 4 (h step)^2, and |step| <= 2.
        assert float(step.abs().max()) <= 2 or name != "dlam"
        tol = (tol_rows(dt) if name in ("dq", "dk", "dv") else tol_acc(dt)) + (16 * h * h if name == "dlam" else 1e-9)
        assert abs((up - down) / (2 * h) - mine) <= tol * size, (name, (up - down) / (2 * h), mine, size)
