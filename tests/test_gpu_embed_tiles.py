"""The table's gradient over tiles of every length.  g holds small whole numbers,
so the sums in fp32 are exact in any order and the result has to be equal: a part
of a run left out, or added twice, shows.

A tile has 16 to 256 sorted positions, doubled while there are more than 148 x 64
warps of 512-byte columns: TILES names a size for each."""
import pytest
import torch

from exact_laplace_b200 import laplex as X

pytestmark = pytest.mark.gpu

BF, HF, F4, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float64
TILES = {16: (9000, 520, BF), 32: (65536, 1024, BF), 64: (65536, 2048, BF), 128: (65536, 4096, BF), 256: (65536, 4096, F4)}


def tile_of(n, dim, es):
    cols, R = max(1, (dim * es + 511) // 512), 16
    while R < 256 and n * cols / R > 148 * 64:
        R *= 2
    return R


def whole(n, dim, dt, seed=0):
    return torch.randint(-4, 5, (n, dim), generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dt)


def want_of(tok, g, rows, old=None):
    """Exact: at most n 4 < 2^24 a sum."""
    known = (tok >= 0) & (tok < rows)
    out = torch.zeros(rows, g.shape[1], device="cuda") if old is None else old.float()
    for a in range(0, g.shape[1], 512):
        out[:, a:a + 512].index_add_(0, tok[known], g[known, a:a + 512].float())
    return out


def runs(n, R, seed):
    """Sorted runs whose ends lie around multiples of R, with up to 40 tiles between, shuffled."""
    gen = torch.Generator().manual_seed(seed)
    ends, at, i = [0], 0, 0
    gaps, offs = [1, 2, 3, 15, 16, 17, 18, 40], [-1, 0, 1, 15, 16, 17]
    while at < n:
        tile = at // R + gaps[i % len(gaps)]
        at = min(n, max(at + 1, tile * R + offs[i // len(gaps) % len(offs)]))
        ends.append(at)
        if i % 3 == 0 and at < n:  # and a short run between
            at += 1
            ends.append(at)
        i += 1
    lens = torch.tensor([b - a for a, b in zip(ends, ends[1:])])
    rows = 2 * len(lens) + 3
    tok = torch.repeat_interleave(2 * torch.arange(len(lens)) + 1, lens)
    return tok[torch.randperm(n, generator=gen)].cuda(), rows


@pytest.mark.parametrize("R", list(TILES))
@pytest.mark.parametrize("out", ["own", "fp32"])
def test_runs_around_tiles(R, out):
    n, dim, dt = TILES[R]
    assert tile_of(n, dim, torch.finfo(dt).bits // 8) == R
    tok, rows = runs(n, R, R)
    g = whole(n, dim, dt)
    want = want_of(tok, g, rows)
    got = X.embed_backward(tok, g, rows, dtype=F4 if out == "fp32" else None)
    assert torch.equal(got, want.to(got.dtype))
    assert torch.equal(X.embed_backward(tok, g, rows, dtype=got.dtype), got)


@pytest.mark.parametrize("n,dim,dt", [(65536, 1024, HF), (65536, 520, F8), (140000, 2048, BF), (300000, 72, F4), (65537, 40, BF),
                                      (200000, 33, HF)], ids=str)
@pytest.mark.parametrize("accumulate", [False, True])
def test_other_types_more_tokens_and_sums(n, dim, dt, accumulate):
    R = tile_of(n, dim, torch.finfo(dt).bits // 8)
    tok, rows = runs(n, R, 1)
    tok[torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) < 0.05] = -1
    g = whole(n, dim, dt)
    to = F8 if dt == F8 else F4
    old = whole(rows, dim, to, 5)
    want = want_of(tok, g, rows, old if accumulate else None)
    out = old if accumulate else torch.full((rows, dim), 9.0, dtype=to, device="cuda")
    X.embed_backward(tok, g, rows, out=out, accumulate=accumulate)
    assert torch.equal(out, want.to(to))


@pytest.mark.parametrize("rows", [1, 2, 31, 1024, 1025, 70000, (1 << 20) + 1])
@pytest.mark.parametrize("n", [65535, 65536, 65537])
def test_tables_of_one_to_three_digits(rows, n):
    """The cluster's sort takes 1 to 3 digits by the table's rows; one token more goes another way."""
    gen = torch.Generator("cuda").manual_seed(rows)
    tok = (rows ** torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)).long() - 1
    g = whole(n, 16, BF)
    got = X.embed_backward(tok, g, rows, dtype=F4)
    assert torch.equal(got, want_of(tok, g, rows))
