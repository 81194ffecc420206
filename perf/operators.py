"""Workloads of the sequence operators of exact_laplace_b200, for timing and for
checking: decayed linear attention (a packed batch of prompts, single tokens
against a cache of states, the backward pass) and the embedding lookup with its
gradient.

`run` computes an operator from elementary torch operations in 32 bits, rounded
once at the end, or, with `own` set, by the calls that a user makes of
exact_laplace_b200.laplex.  `exact` restates each operator's definition in 64
bits.

    linattn          S_t = e^lam S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t, per
                     sequence and head (lam: the head's log decay; a group of
                     query heads shares its k/v head's state)
    linattn_step     the same for one token per row of a cache of states, in place
    linattn_backward gradients of <do, o> + <dS, S_last>
    embed            out_i = scale table[token_i] (zeros for a token out of range)
    embed_backward   dW_r = scale sum over {i: token_i = r} of g_i
"""
import math
import random

import torch

own = False

C = 128  # tokens per block of the plain form
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ----------------------------------------------------------------------------- cases

def _att(op, dtype, tokens, seqs, hq, hkv, dk, dv, ragged, state):
    return {"op": op, "dtype": dtype, "tokens": tokens, "seqs": seqs, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv,
            "ragged": ragged, "state": state}


def _step(dtype, rows, slots, hq, hkv, dk, dv):
    return {"op": "step", "dtype": dtype, "rows": rows, "slots": slots, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv}


def _emb(op, dtype, tokens, rows, dim, padded):
    return {"op": op, "dtype": dtype, "tokens": tokens, "rows": rows, "dim": dim, "padded": padded}


def listed():
    return [
        # one short prompt of a small model, its state kept for the tokens to come: latency
        dict(_att("forward", "bf16", 200, 1, 8, 8, 64, 64, False, True), name="forward short prompt bf16"),
        # a packed batch of prompts of different lengths, four query heads to a k/v head
        dict(_att("forward", "fp16", 16384, 24, 32, 8, 128, 128, True, True), name="forward packed grouped fp16"),
        # one long document, continued from a state
        dict(_att("forward", "bf16", 65536, 1, 16, 16, 128, 128, False, True), name="forward long bf16"),
        # the same operator in the library's own type, head sizes that fill no tile
        dict(_att("forward", "fp32", 6000, 5, 6, 6, 72, 104, True, True), name="forward ragged fp32"),
        # one user's next token
        dict(_step("bf16", 1, 4, 16, 16, 128, 128), name="step one bf16"),
        # a full serving batch over a cache of states
        dict(_step("bf16", 256, 300, 32, 16, 128, 128), name="step batch bf16"),
        # a small training batch, head sizes that differ
        dict(_att("backward", "fp16", 1500, 3, 4, 4, 64, 96, True, False), name="backward small fp16"),
        # a training batch of long sequences
        dict(_att("backward", "bf16", 32768, 4, 16, 16, 128, 128, False, False), name="backward long bf16"),
        # tokens of one serving step
        dict(_emb("embed", "fp32", 96, 32768, 1024, False), name="embed step fp32"),
        # tokens of a training batch
        dict(_emb("embed", "bf16", 65536, 131072, 4096, True), name="embed batch bf16"),
        # the gradient of a small table
        dict(_emb("embed_backward", "fp32", 4000, 8192, 520, False), name="embed backward small fp32"),
        # the gradient of a large one: frequent tokens take thousands of rows, most take none
        dict(_emb("embed_backward", "bf16", 65536, 131072, 2048, True), name="embed backward large bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "step", "backward", "embed", "embed_backward"])
    dtype = rng.choice(["bf16", "fp16", "fp32"] if op in ("embed", "embed_backward") else ["bf16", "bf16", "fp16", "fp32"])
    if op in ("forward", "backward"):
        hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
        hq = hkv * rng.choice([1, 1, 2, 4])
        most = (1 << 20) // hq if op == "forward" else (1 << 19) // hq
        tokens = _log(rng, 1, min(65536, most))
        return _att(op, dtype, tokens, _log(rng, 1, min(32, tokens)), hq, hkv, 8 * rng.randint(2, 16), 8 * rng.randint(2, 16),
                    rng.random() < 0.7, rng.random() < 0.5)
    if op == "step":
        rows = _log(rng, 1, 256)
        hkv = rng.choice([1, 2, 4, 8, 16])
        return _step(dtype, rows, rows + rng.randint(0, 40), hkv * rng.choice([1, 2]), hkv, 8 * rng.randint(2, 16), 8 * rng.randint(2, 16))
    dim = 8 * _log(rng, 8, 512)
    tokens = _log(rng, 1, 65536)
    rows = _log(rng, 100, 131072)
    if op == "embed_backward" and rows * dim > 131072 * 2048:
        dim = max(8, 131072 * 2048 // rows // 8 * 8)
    if (tokens + rows) * dim > 500_000_000:
        tokens = max(1, min(tokens, 65536 * 2048 // dim))
    return _emb(op, dtype, tokens, rows, dim, rng.random() < 0.5)


def work(case):
    s = SIZE[case["dtype"]]
    if case["op"] in ("embed", "embed_backward"):
        n, d = case["tokens"], case["dim"]
        # the lookup writes a row per token and reads no row of the table twice; the gradient reads a row per
        # token and writes the table's
        return {"bytes": 4 * n + s * d * (n + (min(n, case["rows"]) if case["op"] == "embed" else case["rows"])), "flops": n * d}
    hq, hkv, dk, dv = (case[x] for x in ("hq", "hkv", "dk", "dv"))
    if case["op"] == "step":
        n = case["rows"]
        return {"bytes": n * (s * (hq + hkv) * (dk + dv) + 8 * hkv * dk * dv), "flops": n * dk * dv * (3 * hkv + 2 * hq)}
    t = case["tokens"]
    states = 4 * case["seqs"] * hkv * dk * dv * (2 if case["state"] else 0)
    once, flops = s * t * (hq + hkv) * (dk + dv), t * dk * dv * (2 * hkv + 2 * hq)
    if case["op"] == "forward":
        return {"bytes": once + states, "flops": flops}
    # reads q, k, v, do; writes dq, dk, dv
    return {"bytes": s * t * (hq * (2 * dk + dv) + 2 * hkv * (dk + dv)) + states, "flops": 3 * flops}


# ----------------------------------------------------------------------------- inputs

def _lengths(case, seed):
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        base, more = divmod(t, n)
        return [base + (1 if i < more else 0) for i in range(n)]
    rng = random.Random(seed * 7919 + 17)
    cuts = [0] + sorted(rng.randint(0, t) for _ in range(n - 1)) + [t]  # short, long and empty sequences
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _decays(heads, dev):
    # from about 8 to about 2000 tokens of memory, spread over the heads
    mem = 8.0 * (250.0 ** (torch.arange(heads, dtype=torch.float64) / max(heads - 1, 1)))
    return torch.log1p(-1.0 / mem).float().to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 12345)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    if case["op"] in ("embed", "embed_backward"):
        n, rows, dim = case["tokens"], case["rows"], case["dim"]
        # Zipf: the rank's density falls as 1 / rank; ranks lie scattered over the ids
        u = torch.rand(n, generator=g, device=dev, dtype=torch.float64)
        rank = (torch.exp(u * math.log(rows)) - 1).long().clamp_(0, rows - 1)
        step = 48271
        while math.gcd(step, rows) != 1:
            step += 2
        tok = ((rank * step + 11) % rows).to(torch.int32)
        if case["padded"]:  # the padding of a batch: no row
            tok = torch.where(torch.rand(n, generator=g, device=dev) < 0.1, torch.full_like(tok, -1), tok)
        st = {"case": case, "tokens": tok, "scale": math.sqrt(dim)}
        if case["op"] == "embed":
            st["table"] = normal(rows, dim)
        else:
            st["g"] = normal(n, dim)
        return st
    hq, hkv, dk, dv = (case[x] for x in ("hq", "hkv", "dk", "dv"))
    st = {"case": case, "lam": _decays(hkv, dev), "scale": dk ** -0.5}
    if case["op"] == "step":
        n = case["rows"]
        st.update(q=normal(n, hq, dk), k=normal(n, hkv, dk), v=normal(n, hkv, dv),
                  states=3.0 * normal(case["slots"], hkv, dk, dv, dtype=torch.float32),
                  slots=torch.randperm(case["slots"], generator=g, device=dev)[:n].to(torch.int32))
        return st
    lens = _lengths(case, seed)
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
    t = case["tokens"]
    # q, k and v as the projection of the layer leaves them: slices of one row
    if hq * dk % 8 == 0 and hkv * dk % 8 == 0:
        row = normal(t, hq * dk + hkv * dk + hkv * dv)
        q, k, v = row.split([hq * dk, hkv * dk, hkv * dv], 1)
    else:
        q, k, v = normal(t, hq * dk), normal(t, hkv * dk), normal(t, hkv * dv)
    st.update(q=q.view(t, hq, dk), k=k.view(t, hkv, dk), v=v.view(t, hkv, dv), lens=lens, cu=cu.to(dev),
              state=3.0 * normal(case["seqs"], hkv, dk, dv, dtype=torch.float32) if case["state"] else None)
    if case["op"] == "backward":
        st["do"] = normal(t, hq, dv)
        st["dstate"] = 3.0 * normal(case["seqs"], hkv, dk, dv, dtype=torch.float32) if case["state"] else None
    return st


# ----------------------------------------------------------------------------- the plain form

class _Blocks:
    """Tokens of the packed sequences in blocks of at most C of one sequence."""

    def __init__(self, lens, cu, lam):
        dev = lam.device
        n = len(lens)
        count = torch.tensor([-(-x // C) for x in lens], device=dev)
        blocks = sum(-(-x // C) for x in lens)
        self.seq = torch.repeat_interleave(torch.arange(n, device=dev), count, output_size=blocks)
        first = count.cumsum(0) - count
        self.start = (torch.arange(blocks, device=dev) - first[self.seq]) * C  # position in the sequence
        size = (cu[1:] - cu[:-1]).long()
        self.end = torch.minimum(self.start + C, size[self.seq])
        pos = torch.arange(C, device=dev)
        self.at = cu[:-1].long()[self.seq][:, None] + self.start[:, None] + pos
        self.valid = self.start[:, None] + pos < self.end[:, None]
        self.at = torch.where(self.valid, self.at, torch.zeros_like(self.at))
        self.size, self.n, self.blocks, self.lam = size, n, blocks, lam
        d = (pos[:, None] - pos[None, :]).float()
        self.low = torch.where(d >= 0, torch.exp(lam[:, None, None] * d.clamp(min=0)), torch.zeros((), device=dev))  # [H, t, s]

    def take(self, x):
        """[T, H, D] to [blocks, H, C, D], zeros where a block has no token."""
        return torch.where(self.valid[..., None, None], x[self.at].float(), torch.zeros((), device=x.device)).transpose(1, 2)

    def put(self, x, like):
        """[blocks, H, C, D] back to [T, H, D], in like's type."""
        out = torch.zeros(like.shape, dtype=torch.float32, device=x.device)
        out[self.at[self.valid]] = x.transpose(1, 2)[self.valid]
        return out.to(like.dtype)

    def weight(self, far, known):
        """exp(lam far) where known, [H, ...]"""
        lam = self.lam.view(-1, *([1] * far.dim()))
        return torch.where(known, torch.exp(lam * torch.where(known, far, torch.zeros_like(far)).float()), torch.zeros((), device=far.device))


def _attention(b, q, k, v, state, scale, last):
    """Blocks q [blocks, H, G, C, dk], k, v [blocks, H, C, d] -> o, and the last states where asked."""
    pos = torch.arange(C, device=q.device)
    size = b.end - b.start
    left = (size[:, None] - 1 - pos).clamp(min=0)
    part = torch.einsum("bhsd,bhse->hbde", k * b.weight(left, b.valid).transpose(0, 1)[..., None], v)
    same = b.seq[:, None] == b.seq[None, :]
    gap = b.start[:, None] - b.end[None, :]
    dk, dv = k.shape[-1], v.shape[-1]
    before = (b.weight(gap, same & (gap >= 0)) @ part.flatten(2)).unflatten(2, (dk, dv))
    if state is not None:
        before = before + b.weight(b.start, b.start >= 0)[..., None, None] * state[b.seq].transpose(0, 1)
    score = torch.einsum("bhgtd,bhsd->bhgts", q, k) * b.low[:, None]
    o = score @ v[:, :, None]
    o = o + torch.einsum("bhgtd,hbde->bhgte", q, before) * torch.exp(b.lam[:, None, None] * (pos + 1.0))[..., None]
    end = None
    if last:
        tail = b.size[:, None] - b.end[None, :]
        mine = torch.arange(b.n, device=q.device)[:, None] == b.seq[None, :]
        end = (b.weight(tail, mine) @ part.flatten(2)).unflatten(2, (dk, dv)).transpose(0, 1)
        if state is not None:
            end = end + torch.exp(b.lam * b.size[:, None].float())[..., None, None] * state
    return scale * o, end


def _forward(st):
    q, k, v = st["q"], st["k"], st["v"]
    b = _Blocks(st["lens"], st["cu"], st["lam"])
    h = k.shape[1]
    o, end = _attention(b, b.take(q).unflatten(1, (h, -1)), b.take(k), b.take(v), st["state"], st["scale"], True)
    return {"o": b.put(o.flatten(1, 2), torch.empty((*q.shape[:2], v.shape[2]), dtype=q.dtype, device="meta")), "state": end}


def _backward(st):
    q, k, v, do, s0, ds, scale = (st[x] for x in ("q", "k", "v", "do", "state", "dstate", "scale"))
    b = _Blocks(st["lens"], st["cu"], st["lam"])
    h = k.shape[1]
    qb, kb, vb, dob = b.take(q).unflatten(1, (h, -1)), b.take(k), b.take(v), b.take(do).unflatten(1, (h, -1))
    # dq is the same product with the parts exchanged: do against v, summing k
    dq, _ = _attention(b, dob, vb, kb, None if s0 is None else s0.transpose(2, 3), scale, False)
    # the states' gradient, from the blocks behind
    pos = torch.arange(C, device=q.device)
    up = b.weight(pos.expand(b.blocks, C) + 1, b.valid).transpose(0, 1)  # to the block's start
    part = scale * torch.einsum("bhgtd,bhgte->hbde", qb * up[:, :, None, :, None], dob)
    same = b.seq[:, None] == b.seq[None, :]
    gap = b.start[None, :] - b.end[:, None]
    dk_, dv_ = k.shape[-1], v.shape[-1]
    after = (b.weight(gap, same & (gap >= 0)) @ part.flatten(2)).unflatten(2, (dk_, dv_))
    if ds is not None:
        after = after + b.weight(b.size[b.seq] - b.end, b.end >= 0)[..., None, None] * ds[b.seq].transpose(0, 1)
    size = b.end - b.start
    left = b.weight((size[:, None] - 1 - pos).clamp(min=0), b.valid).transpose(0, 1)[..., None]
    score = torch.einsum("bhgtd,bhsd->bhgts", qb, kb) * b.low[:, None]
    dscore = torch.einsum("bhgte,bhse->bhgts", dob, vb) * b.low[:, None]
    dv = scale * torch.einsum("bhgts,bhgte->bhse", score, dob) + left * torch.einsum("bhsd,hbde->bhse", kb, after)
    dk = scale * torch.einsum("bhgts,bhgtd->bhsd", dscore, qb) + left * torch.einsum("bhse,hbde->bhsd", vb, after)
    out = {"dq": b.put(dq.flatten(1, 2), q), "dk": b.put(dk, k), "dv": b.put(dv, v)}
    if s0 is not None:
        mine = torch.arange(b.n, device=q.device)[:, None] == b.seq[None, :]
        first = (b.weight(b.start.expand(b.n, -1), mine) @ part.flatten(2)).unflatten(2, (dk_, dv_)).transpose(0, 1)
        out["dstate"] = first + torch.exp(b.lam * b.size[:, None].float())[..., None, None] * ds
    return out


def _one_token(st):
    q, k, v, lam, at = st["q"], st["k"], st["v"], st["lam"], st["slots"].long()
    new = torch.exp(lam)[:, None, None] * st["states"][at] + k.float()[..., None] * v.float()[:, :, None]
    st["states"][at] = new
    o = st["scale"] * torch.einsum("nhgd,nhde->nhge", q.float().unflatten(1, (k.shape[1], -1)), new)
    return {"o": o.flatten(1, 2).to(q.dtype), "states": st["states"]}


def _embed(st):
    tok, table = st["tokens"].long(), st["table"]
    known = (tok >= 0) & (tok < table.shape[0])
    rows = table[torch.where(known, tok, torch.zeros_like(tok))].float() * st["scale"]
    return torch.where(known[:, None], rows, torch.zeros((), device=rows.device)).to(table.dtype)


def _embed_backward(st):
    tok, g, rows = st["tokens"].long(), st["g"], st["case"]["rows"]
    known = (tok >= 0) & (tok < rows)
    out = torch.zeros(rows + 1, g.shape[1], device=g.device)
    out.index_add_(0, torch.where(known, tok, torch.full_like(tok, rows)), g.float())
    return (out[:rows] * st["scale"]).to(g.dtype)


def run(st):
    op = st["case"]["op"]
    if own:
        from exact_laplace_b200 import laplex as X
        if op == "forward":
            o, end = X.linattn(st["q"], st["k"], st["v"], st["lam"], scale=st["scale"], cu_seqlens=st["cu"], state=st["state"],
                               return_state=True)
            return {"o": o, "state": end}
        if op == "backward":
            g = X.linattn_backward(st["q"], st["k"], st["v"], st["lam"], st["do"], scale=st["scale"], cu_seqlens=st["cu"],
                                   state=st["state"], dstate=st["dstate"])
            out = {"dq": g.dq, "dk": g.dk, "dv": g.dv}
            return out if st["state"] is None else dict(out, dstate=g.dstate)
        if op == "step":
            o = X.linattn_step(st["q"], st["k"], st["v"], st["lam"], st["states"], slots=st["slots"], scale=st["scale"])
            return {"o": o, "states": st["states"]}
        if op == "embed":
            return X.embed(st["table"], st["tokens"], scale=st["scale"])
        return X.embed_backward(st["tokens"], st["g"], st["case"]["rows"], scale=st["scale"])
    return {"forward": _forward, "backward": _backward, "step": _one_token, "embed": _embed, "embed_backward": _embed_backward}[op](st)


# ----------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f = torch.float64
    if case["op"] == "embed":
        table = st["table"].to(f)
        table = torch.cat([table * st["scale"], torch.zeros_like(table[:1])])
        tok = st["tokens"].long()
        return table[torch.where(tok < 0, torch.full_like(tok, case["rows"]), tok)]
    if case["op"] == "embed_backward":
        out = torch.zeros(case["rows"], case["dim"], dtype=f, device="cuda")
        keep = st["tokens"] >= 0
        tok = st["tokens"][keep].long()
        for a in range(0, case["dim"], 512):
            out[:, a:a + 512].index_add_(0, tok, st["g"][keep, a:a + 512].to(f))
        return out * st["scale"]
    lam = st["lam"].to(f)
    group = case["hq"] // case["hkv"]
    if case["op"] == "step":
        states, o = st["states"].to(f), []
        for r, slot in enumerate(st["slots"].tolist()):
            states[slot] = torch.exp(lam)[:, None, None] * states[slot] + st["k"][r].to(f)[:, :, None] * st["v"][r].to(f)[:, None, :]
            read = states[slot].repeat_interleave(group, 0)
            o.append(st["scale"] * (st["q"][r].to(f)[:, :, None] * read).sum(1))
        return {"o": torch.stack(o), "states": states}
    back = case["op"] == "backward"
    scale, s0 = st["scale"], st["state"]
    t = case["tokens"]
    res = {"o": torch.zeros(t, case["hq"], case["dv"], dtype=f, device="cuda")}
    if back:
        res = {"dq": torch.zeros(t, case["hq"], case["dk"], dtype=f, device="cuda"),
               "dk": torch.zeros(t, case["hkv"], case["dk"], dtype=f, device="cuda"),
               "dv": torch.zeros(t, case["hkv"], case["dv"], dtype=f, device="cuda")}
    end = torch.zeros(case["seqs"], case["hkv"], case["dk"], case["dv"], dtype=f, device="cuda")
    a = 0
    for n, length in enumerate(st["lens"]):
        at = torch.arange(length, device="cuda", dtype=f)
        for h in range(case["hkv"]):
            k, v = st["k"][a:a + length, h].to(f), st["v"][a:a + length, h].to(f)
            keep = torch.exp(lam[h] * length)
            init = None if s0 is None else s0[n, h].to(f)
            if back:
                if init is not None:
                    end[n, h] = keep * st["dstate"][n, h].to(f)
            else:
                end[n, h] = (torch.exp(lam[h] * (length - 1 - at))[:, None] * k).T @ v + (0 if init is None else keep * init)
            for i in range(h * group, (h + 1) * group):
                q = st["q"][a:a + length, i].to(f)
                do = st["do"][a:a + length, i].to(f) if back else None
                for r in range(0, length, 2048):  # rows of the dense, lower triangular kernel
                    s = min(r + 2048, length)
                    far = at[r:s, None] - at[None, :s]
                    w = scale * torch.where(far >= 0, torch.exp(lam[h] * far.clamp(min=0)), torch.zeros((), dtype=f, device="cuda"))
                    lead = torch.exp(lam[h] * (at[r:s] + 1))[:, None]
                    p = (q[r:s] @ k[:s].T) * w
                    if not back:
                        res["o"][a + r:a + s, i] = p @ v[:s] + (0 if init is None else scale * lead * (q[r:s] @ init))
                        continue
                    dp = (do[r:s] @ v[:s].T) * w
                    res["dq"][a + r:a + s, i] = dp @ k[:s] + (0 if init is None else scale * lead * (do[r:s] @ init.T))
                    res["dk"][a:a + s, h] += dp.T @ q[r:s]
                    res["dv"][a:a + s, h] += p.T @ do[r:s]
                if back and init is not None:
                    end[n, h] += scale * (torch.exp(lam[h] * (at + 1))[:, None] * q).T @ do
            if back and init is not None:
                tail = torch.exp(lam[h] * (length - 1 - at))[:, None]
                res["dk"][a:a + length, h] += tail * (v @ st["dstate"][n, h].to(f).T)
                res["dv"][a:a + length, h] += tail * (k @ st["dstate"][n, h].to(f))
        a += length
    if not back:
        res["state"] = end
    elif s0 is not None:
        res["dstate"] = end
    return res
