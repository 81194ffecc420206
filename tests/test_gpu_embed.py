"""Embedding lookup and its gradient on the GPU against their definitions.

Tolerances: the lookup is one product and one rounding, at most half a step of
the type (fp32 and fp64 tables: the product's own rounding).  The gradient of m
rows is summed in the accumulator's type, at most m + 1 roundings of eps_acc / 2
of the sum of magnitudes, then rounded once to the table's type.
"""
import numpy as np
import pytest
import torch

from exact_laplace_b200 import laplex as X
from oracle import seq

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp64": torch.float64}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def np64(t):
    return t.detach().cpu().double().numpy()


def values(shape, dt, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).to(dt).cuda()


def tokens(kind, n, rows, seed=0):
    rng = np.random.default_rng(seed + n)
    if kind == "uniform":
        t = rng.integers(0, rows, n)
    elif kind == "zipf":
        t = np.minimum((rows ** rng.random(n)).astype(np.int64) - 1, rows - 1) * 7919 % rows
    elif kind == "one":
        t = np.full(n, rows - 1)
    elif kind == "padded":
        t = rng.integers(-2, rows + 2, n)
        t[rng.random(n) < 0.2] = -1
    elif kind == "none":
        t = np.full(n, -100)
    else:
        t = np.arange(n) % rows
    return t


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("dim", [1, 7, 8, 64, 520, 1000, 2051])
@pytest.mark.parametrize("wide", [False, True])
def test_lookup(dt, dim, wide):
    rows = 37
    table = values((rows, dim + 8), DT[dt], dim)[:, :dim] if wide else values((rows, dim), DT[dt], dim)
    for n in (1, 5, 33, 200):
        t = tokens("padded", n, rows)
        want = seq.embed(np64(table), t, 1.7)
        for it in (torch.int32, torch.int64):
            got = X.embed(table, torch.from_numpy(t).to(it).cuda(), scale=1.7)
            # 1.7 itself is rounded to fp32: one half step of fp32 more
            u = half_step(DT[dt]) + (half_step(torch.float32) if dt != "fp64" else half_step(torch.float64)) * 2
            assert np.all(np.abs(np64(got) - want) <= u * np.abs(want) * (1 + 1e-6) + 2.0 ** -25 * (dt == "fp16"))
            assert np.all(np64(got)[(t < 0) | (t >= rows)] == 0)


def test_lookup_keeps_shapes_and_nan_rows():
    table = values((9, 24), torch.bfloat16, 0)
    table[4] = float("nan")
    t = torch.tensor([[4, 1, 1], [-1, 8, 2 ** 40]], device="cuda")
    o = X.embed(table, t, scale=float("inf"))
    assert o.shape == (2, 3, 24) and torch.isnan(o[0, 0]).all()
    assert torch.all(o[1, 0] == 0) and torch.all(o[1, 2] == 0)  # no row, not 0 * inf
    out = torch.full((2, 3, 24), 3.0, dtype=torch.bfloat16, device="cuda")
    assert X.embed(table, t, out=out) is out and torch.equal(out[0, 1], table[1])
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    assert X.embed(table, empty).shape == (0, 24)


def check_gradient(got, t, g, rows, scale, dt, out_dt, old=None):
    want = seq.embed_backward(t, np64(g), rows, scale)
    mag = seq.embed_backward(t, np.abs(np64(g)), rows, abs(scale))
    m = max(np.bincount(t[(t >= 0) & (t < rows)], minlength=rows).max(initial=0), 1)
    if old is not None:
        want, mag = want + np64(old), mag + np.abs(np64(old))
    ua = half_step(torch.float64 if dt == torch.float64 else torch.float32)
    tol = (m + 3) * ua * mag + half_step(out_dt) * (1 + (m + 3) * ua) * np.abs(want)
    # a value below the 16-bit type's normal range is rounded on its smallest step
    tol = tol + (2.0 ** -25 if out_dt == torch.float16 else 0)
    bad = np.abs(np64(got) - want) > tol
    assert not bad.any(), (bad.sum(), np.abs(np64(got) - want).max())


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("kind", ["uniform", "zipf", "one", "padded", "none", "cycle"])
def test_gradient(dt, kind):
    for n, rows, dim in ((1, 5, 8), (15, 3, 64), (16, 40, 24), (17, 1, 33), (300, 64, 72), (5000, 700, 40), (9000, 2, 8)):
        t = tokens(kind, n, rows)
        g = values((n, dim), DT[dt], n)
        for it in (torch.int32, torch.int64):
            got = X.embed_backward(torch.from_numpy(t).to(it).cuda(), g, rows, scale=0.75)
            check_gradient(got, t, g, rows, 0.75, DT[dt], DT[dt])


@pytest.mark.parametrize("n,rows,dim", [(1, 70000, 8), (20000, 100000, 16), (70000, 300, 8), (40000, 1 << 17, 264),
                                        (200000, 66000, 8)])
def test_gradient_sizes(n, rows, dim):
    t = tokens("zipf", n, rows)
    g = values((n, dim), torch.bfloat16, n)
    got = X.embed_backward(torch.from_numpy(t).cuda(), g, rows, dtype=torch.float32)
    check_gradient(got, t, g, rows, 1.0, torch.bfloat16, torch.float32)
    assert torch.equal(got, X.embed_backward(torch.from_numpy(t).cuda(), g, rows, dtype=torch.float32))


@pytest.mark.parametrize("dt", ["bf16", "fp32", "fp64"])
@pytest.mark.parametrize("dim", [8, 130, 264])
def test_gradient_of_runs_around_the_tiles(dt, dim):
    # runs that begin and end around multiples of 16 positions, with 1 to 1300 tiles between
    lens = [16 * k + d for k in (1, 2, 15, 16, 17, 18, 33) for d in (-1, 0, 1, 15)] + [20800]
    rng = np.random.default_rng(7)
    n, rows = sum(lens), 3 * len(lens)
    t = np.repeat(3 * rng.permutation(len(lens)), lens)[rng.permutation(n)]
    g = values((n, dim), DT[dt], 8)
    got = X.embed_backward(torch.from_numpy(t).cuda(), g, rows, scale=0.5)
    check_gradient(got, t, g, rows, 0.5, DT[dt], DT[dt])
    assert torch.equal(got, X.embed_backward(torch.from_numpy(t).cuda(), g, rows, scale=0.5))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,dim,ld", [(300, 64, 72), (300, 64, 67), (90000, 512, 520), (33, 8, 8)])
def test_gradient_into_a_part_of_wider_rows(dt, rows, dim, ld):
    # rows zeroed beside the sort, and those zeroed beside the sums
    t = tokens("padded", 2000, rows)
    g = values((2000, dim), DT[dt], 6)
    whole = torch.full((rows + 2, ld), 7.0, dtype=DT[dt], device="cuda")
    out = whole[:rows, :dim]
    X.embed_backward(torch.from_numpy(t).cuda(), g, rows, out=out)
    check_gradient(out, t, g, rows, 1.0, DT[dt], DT[dt])
    assert bool((whole[rows:] == 7).all()) and bool((whole[:, dim:] == 7).all())


@pytest.mark.parametrize("dt,out_dt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp32"), ("fp32", "fp32"), ("fp64", "fp64")])
def test_gradient_accumulates(dt, out_dt):
    n, rows, dim = 700, 90, 40
    t = tokens("padded", n, rows)
    t[t == 3] = -1  # a row that no token names
    g = values((n, dim), DT[dt], 1)
    out = values((rows, dim), DT[out_dt], 2)
    out[3] = float("nan")
    old = out.clone()
    assert X.embed_backward(torch.from_numpy(t).cuda(), g, rows, scale=-2.0, out=out, accumulate=True) is out
    assert torch.isnan(out[3]).all()
    keep = [i for i in range(rows) if i != 3]
    old[3] = 0
    out[3] = 0
    check_gradient(out[keep], np.where(t > 3, t - 1, t), g, rows - 1, -2.0, DT[dt], DT[out_dt], old[keep])


def test_gradient_of_strided_rows_and_nan_padding():
    """Rows of padding tokens are not read; dtable inside a wider buffer."""
    n, rows, dim = 500, 60, 48
    t = tokens("padded", n, rows)
    wide = values((n, dim + 16), torch.bfloat16, 3)
    g = wide[:, 8:8 + dim]
    g[torch.from_numpy((t < 0) | (t >= rows)).cuda()] = float("nan")
    buf = torch.full((rows, dim + 8), 9.0, dtype=torch.float32, device="cuda")
    X.embed_backward(torch.from_numpy(t).cuda(), g, rows, out=buf[:, :dim])
    clean = torch.nan_to_num(g)
    check_gradient(buf[:, :dim], t, clean, rows, 1.0, torch.bfloat16, torch.float32)
    assert torch.all(buf[:, dim:] == 9)


def test_gradient_in_a_graph():
    n, rows, dim = 3000, 500, 64
    t = torch.from_numpy(tokens("zipf", n, rows)).cuda()
    g = values((n, dim), torch.bfloat16, 5)
    want = X.embed_backward(t, g, rows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = X.embed_backward(t, g, rows)
        rows_out = X.embed(got, t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(rows_out, X.embed(want, t))
    t.copy_(t.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, X.embed_backward(t, g, rows))


def test_empty():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    g = torch.empty((0, 16), device="cuda")
    assert torch.all(X.embed_backward(none, g, 5) == 0)
    assert X.embed_backward(none, g, 0).shape == (0, 16)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_tokens_past_32_bits_are_outside(dt):
    table = values((40, 64), DT[dt], 1)
    t = torch.tensor([3, 2 ** 32 + 3, -2 ** 32 + 3, 2 ** 63 - 1, -2 ** 63, 39, 40], dtype=torch.int64, device="cuda")
    out = X.embed(table, t)
    want = torch.zeros_like(out)
    want[0], want[5] = table[3], table[39]
    assert torch.equal(out, want)
    g = values((7, 64), DT[dt], 2)
    d = X.embed_backward(t, g, 40)
    want = torch.zeros_like(table)
    want[3], want[39] = g[0], g[5]
    assert torch.equal(d, want)


def test_table_past_32_bits():
    rows, dim = (1 << 21) + 5, 1032  # 2.16e9 elements
    if torch.cuda.mem_get_info()[0] < 4 * rows * dim * 2:
        pytest.skip("not enough memory")
    table = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    t = torch.tensor([rows - 1, 0, rows - 3, rows - 1], dtype=torch.int32, device="cuda")
    x = values((3, dim), torch.bfloat16, 3)
    table[[rows - 1, 0, rows - 3]] = x
    assert torch.equal(X.embed(table, t), x[[0, 1, 2, 0]])
    table.fill_(1.0)
    d = X.embed_backward(t, x[[0, 1, 2, 0]], rows, out=table)
    assert torch.equal(d[rows - 1], 2 * x[0]) and torch.equal(d[0], x[1]) and torch.equal(d[rows - 3], x[2])
    assert int(torch.count_nonzero(d.view(-1)[:(1 << 20) * dim])) == int(torch.count_nonzero(x[1]))
    assert int(torch.count_nonzero(d[1 << 20:])) == int(torch.count_nonzero(x[0]) + torch.count_nonzero(x[2]))


def test_two_streams_and_two_graphs():
    a = (torch.from_numpy(tokens("zipf", 5000, 700)).cuda(), values((5000, 72), torch.bfloat16, 4), 700)
    b = (torch.from_numpy(tokens("uniform", 90000, 4000)).cuda(), values((90000, 8), torch.bfloat16, 5), 4000)
    want = [X.embed_backward(*x) for x in (a, b)]
    streams, graphs, res = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(X.embed_backward(*x))
        graphs.append(g)
    for _ in range(3):
        eager = []
        for st, g, x in zip(streams, graphs, (b, a)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
                eager.append(X.embed_backward(*x))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, res))
        assert all(torch.equal(x, y) for x, y in zip(want, eager[::-1]))
