"""The fp64 oracle of the sequence operators: hand-worked values, the
recurrence, differences, and the library's own kernel as a special case."""
import numpy as np
import pytest

import oracle as O
from oracle import seq


def rnd(*shape, seed=0):
    return np.random.default_rng(seed + sum(shape)).standard_normal(shape)


def recurrence(q, k, v, lam, scale, lens, state):
    """The states one token at a time."""
    hq, hkv = q.shape[1], k.shape[1]
    o = np.zeros((q.shape[0], hq, v.shape[2]))
    end = np.zeros((len(lens), hkv, q.shape[2], v.shape[2]))
    a = 0
    for n, length in enumerate(lens):
        for h in range(hkv):
            S = np.zeros((q.shape[2], v.shape[2])) if state is None else state[n, h].copy()
            for t in range(a, a + length):
                S = np.exp(lam[h]) * S + np.outer(k[t, h], v[t, h])
                for i in range(h * hq // hkv, (h + 1) * hq // hkv):
                    o[t, i] = scale * S.T @ q[t, i]
            end[n, h] = S
        a += length
    return o, end


def test_hand_worked():
    # e^lam = 1/2, dk = dv = 1: S = 2, 2/2 + 3 = 4, 4/2 + 5 = 7;  o = scale q S
    one = lambda *x: np.array(x, dtype=float).reshape(-1, 1, 1)
    o, end = seq.linattn(one(1, 2, 3), one(2, 3, 5), one(1, 1, 1), [np.log(0.5)], 10.0, [3])
    assert np.allclose(o.ravel(), [20, 80, 210]) and np.allclose(end, 7)
    o, end = seq.linattn(one(1), one(2), one(1), [np.log(0.5)], 1.0, [1], state=np.full((1, 1, 1, 1), 6.0))
    assert np.allclose(o, 5) and np.allclose(end, 5)


@pytest.mark.parametrize("lens", [[7], [3, 0, 1, 5], [0]])
@pytest.mark.parametrize("state", [False, True])
def test_dense_is_the_recurrence(lens, state):
    t, n = sum(lens), len(lens)
    q, k, v = rnd(t, 4, 3), rnd(t, 2, 3, seed=1), rnd(t, 2, 5, seed=2)
    s0 = rnd(n, 2, 3, 5, seed=3) if state else None
    lam = np.array([-0.3, -2.0])
    for got, want in zip(seq.linattn(q, k, v, lam, 0.7, lens, s0), recurrence(q, k, v, lam, 0.7, lens, s0)):
        assert np.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_phased_kernel_is_its_causal_half_with_rank_two():
    """q = (cos phi, sin phi), k = (cos psi, sin psi), anchors -lam t: the causal
    product plus the reversed one, less the diagonal, is the phased product."""
    n, lam = 40, -0.17
    phi, x = rnd(n), rnd(n, seed=5)
    f = np.stack([np.cos(phi), np.sin(phi)], 1)[:, None]
    v = x.reshape(n, 1, 1)
    low = seq.linattn(f, f, v, [lam], 1.0, [n])[0].ravel()
    up = seq.linattn(f[::-1], f[::-1], v[::-1], [lam], 1.0, [n])[0].ravel()[::-1]
    a = -lam * np.arange(n)
    assert np.allclose(low + up - x, O.phased(a, phi, x), rtol=1e-10, atol=1e-12)


def test_gradients_by_differences():
    lens = [4, 0, 1, 3]
    t, n = sum(lens), len(lens)
    args = {"q": rnd(t, 4, 2), "k": rnd(t, 2, 2, seed=1), "v": rnd(t, 2, 3, seed=2), "lam": np.array([-0.4, -1.3]),
            "state": rnd(n, 2, 2, 3, seed=3)}
    do, ds = rnd(t, 4, 3, seed=4), rnd(n, 2, 2, 3, seed=6)

    def loss(a):
        o, end = seq.linattn(a["q"], a["k"], a["v"], a["lam"], 0.6, lens, a["state"])
        return np.sum(o * do) + np.sum(end * ds)

    got = seq.linattn_backward(args["q"], args["k"], args["v"], args["lam"], do, 0.6, lens, args["state"], ds)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("lam", "dlam"), ("state", "dstate")):
        for at in np.ndindex(args[name].shape):
            d = []
            for e in (1e-6, -1e-6):
                b = {x: y.copy() for x, y in args.items()}
                b[name][at] += e
                d.append(loss(b))
            assert abs((d[0] - d[1]) / 2e-6 - got[key][at]) < 1e-7 * (1 + abs(got[key][at])), (name, at)


def test_embedding():
    table = np.arange(6.0).reshape(3, 2)
    tok = np.array([2, -1, 0, 2, 3])
    assert np.array_equal(seq.embed(table, tok, 2.0), [[8, 10], [0, 0], [0, 2], [8, 10], [0, 0]])
    g = np.arange(10.0).reshape(5, 2)
    assert np.array_equal(seq.embed_backward(tok, g, 3, 0.5), [[2, 2.5], [0, 0], [3, 4]])
