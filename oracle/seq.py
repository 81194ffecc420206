"""fp64 statement of the sequence operators, by their definitions (numpy, dense).

linattn: o_t = scale sum_{s <= t} e^{lam (t - s)} <q_t, k_s> v_s + scale e^{lam (t + 1)} S_in^T q_t,
S_out = sum_s e^{lam (L - 1 - s)} k_s v_s^T + e^{lam L} S_in, per sequence and k/v-head.
linattn_backward differentiates those two lines.  embed and embed_backward are
the gather and the scatter-add of rows.
"""
import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _power(lam, d):
    """e^(lam d) with e^(-inf 0) = 1, for d >= 0."""
    d = np.asarray(d, dtype=np.float64)
    return np.where(d == 0, 1.0, np.exp(np.where(d == 0, 0.0, lam) * np.where(d == 0, 1.0, d)))


def _weights(lam, n):
    far = np.arange(n)[:, None] - np.arange(n)[None, :]
    return np.where(far >= 0, _power(lam, np.maximum(far, 0)), 0.0)


def linattn(q, k, v, lam, scale, lens, state=None):
    """(o [T, hq, dv], states [N, hkv, dk, dv]); rows behind the last sequence are 0."""
    q, k, v, lam, state = _f(q), _f(k), _f(v), _f(lam), _f(state)
    hq, hkv, dk, dv = q.shape[1], k.shape[1], q.shape[2], v.shape[2]
    o = np.zeros((q.shape[0], hq, dv))
    end = np.zeros((len(lens), hkv, dk, dv))
    a = 0
    for n, length in enumerate(lens):
        sl = slice(a, a + length)
        for h in range(hkv):
            kk, vv = k[sl, h], v[sl, h]
            with np.errstate(invalid="ignore"):
                end[n, h] = (_power(lam[h], length - 1 - np.arange(length))[:, None] * kk).T @ vv
                if state is not None:
                    end[n, h] += _power(lam[h], length) * state[n, h]
                w = _weights(lam[h], length)
                for i in range(h * hq // hkv, (h + 1) * hq // hkv):
                    o[sl, i] = scale * ((q[sl, i] @ kk.T) * w) @ vv
                    if state is not None:
                        o[sl, i] += scale * _power(lam[h], np.arange(length) + 1)[:, None] * (q[sl, i] @ state[n, h])
        a += length
    return o, end


def linattn_backward(q, k, v, lam, do, scale, lens, state=None, dstate=None):
    """dict of dq, dk, dv, dstate (gradient of `state`), dlam."""
    q, k, v, lam, do, state, dstate = _f(q), _f(k), _f(v), _f(lam), _f(do), _f(state), _f(dstate)
    hq, hkv = q.shape[1], k.shape[1]
    r = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v),
         "dstate": np.zeros((len(lens), hkv, q.shape[2], v.shape[2])), "dlam": np.zeros(hkv)}
    a = 0
    for n, length in enumerate(lens):
        sl = slice(a, a + length)
        at = np.arange(length)
        far = np.maximum(at[:, None] - at[None, :], 0)
        for h in range(hkv):
            kk, vv, w = k[sl, h], v[sl, h], _weights(lam[h], length)
            lead, tail = _power(lam[h], at + 1)[:, None], _power(lam[h], length - 1 - at)[:, None]
            for i in range(h * hq // hkv, (h + 1) * hq // hkv):
                qq, dd = q[sl, i], do[sl, i]
                p, dp = scale * (qq @ kk.T) * w, scale * (dd @ vv.T) * w
                r["dq"][sl, i] = dp @ kk
                r["dk"][sl, h] += dp.T @ qq
                r["dv"][sl, h] += p.T @ dd
                r["dstate"][n, h] += scale * (lead * qq).T @ dd
                r["dlam"][h] += np.sum(far * p * (dd @ vv.T))
                if state is not None:
                    r["dq"][sl, i] += scale * lead * (dd @ state[n, h].T)
                    r["dlam"][h] += scale * np.sum((at + 1)[:, None] * lead * (qq @ state[n, h]) * dd)
            if dstate is not None:
                r["dk"][sl, h] += tail * (vv @ dstate[n, h].T)
                r["dv"][sl, h] += tail * (kk @ dstate[n, h])
                r["dstate"][n, h] += _power(lam[h], length) * dstate[n, h]
                back = length - 1 - at
                r["dlam"][h] += np.sum(back[:, None] * tail * kk * (vv @ dstate[n, h].T))
                if state is not None and length:
                    r["dlam"][h] += length * _power(lam[h], length) * np.sum(state[n, h] * dstate[n, h])
        a += length
    return r


def embed(table, tokens, scale):
    table, tokens = _f(table), np.asarray(tokens)
    known = (tokens >= 0) & (tokens < table.shape[0])
    out = scale * table[np.where(known, tokens, 0)]
    out[~known] = 0.0
    return out


def embed_backward(tokens, g, rows, scale):
    g, tokens = _f(g), np.asarray(tokens)
    out = np.zeros((rows, g.shape[1]))
    known = (tokens >= 0) & (tokens < rows)
    np.add.at(out, tokens[known], scale * g[known])
    return out
