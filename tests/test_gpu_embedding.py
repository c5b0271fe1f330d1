"""Embedding lookup and its gradient on an MI355X against the fp64 oracle.

Forward: one fp32 product, then the result's rounding: equal, bit for bit.
Backward (u = 2^-24): a sum of n terms takes at most n additions one after another
and a product by the scale, (n + 2) u scale sum|dout|, and half a step of the
gradient's type; with accumulate one more addition.
"""

import numpy as np
import pytest
import torch

import pretraining_optimizer_amd as pm
from oracle import embedding
from parity import announce
from sort_plans import SORTS

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


def _tokens(n, rows, kind, seed=0):
    gen = torch.Generator().manual_seed(seed + n)
    if kind == "uniform":
        t = torch.randint(0, max(rows, 1), (n,), generator=gen)
    elif kind == "words":   # a few rows very often
        t = (torch.exp(torch.rand(n, generator=gen, dtype=torch.float64) * np.log(rows + 1)).long() - 1).clamp(0, rows - 1)
    elif kind == "one":
        t = torch.full((n,), rows - 1)
    elif kind == "falling":
        t = (rows - 1 - torch.arange(n) % rows)
    else:                   # some of it padding
        t = torch.randint(0, max(rows, 1), (n,), generator=gen)
        t[::3] = -1
        t[1::7] = rows
    return t


def _check_backward(got, tokens, dout, rows, scale, what, before=None):
    D, t = _np(dout), tokens.cpu().numpy()
    want = embedding.embedding_backward(t, D, rows, scale)
    size = embedding.embedding_backward(t, np.abs(D), rows, abs(scale))
    known = t[(t >= 0) & (t < rows)]
    n = np.bincount(known, minlength=rows)[:rows, None]
    tol = (n + 2) * U * size
    if before is not None:
        want = want + before
        tol = tol + 2 * U * (np.abs(before) + np.abs(want))
    tol = tol + HALF[got.dtype] * (np.abs(want) + tol)
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), (what, float((err - tol).max()))


@pytest.mark.parametrize("table,out", [(F32, BF16), (F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (1, 1000, 2048), (77, 1000, 777), (300, 50, 8), (5, 7, 2049), (1000, 300, 40),
                                         (33, 20, 5000)])
def test_forward(n, rows, cols, table, out):
    announce(f"embedding {n} of {rows}x{cols} {table} {out}")
    weight = torch.randn((rows, cols), generator=torch.Generator().manual_seed(cols)).to(table).cuda()
    for kind, scale in (("uniform", 1.0), ("padding", 45.25)):
        for width in (torch.int64, torch.int32):
            t = _tokens(n, rows, kind).to(width).cuda()
            got = pm.embedding_forward(t, weight, scale=scale, out_dtype=out)
            known = (t >= 0) & (t < rows)
            want = weight[t.long().clamp(0, rows - 1)].float() * torch.tensor(scale, device="cuda")
            want = torch.where(known[:, None], want, torch.zeros_like(want)).to(out)
            assert torch.equal(got, want)
            ref = embedding.embedding_forward(t.tolist(), _np(weight), scale)
            assert np.all(np.abs(_np(got) - ref) <= (U + HALF[out] * (1 + U)) * np.abs(ref))


@pytest.mark.parametrize("dout,table", [(BF16, F32), (F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("n,rows,cols,kind", [
    (1, 1, 1, "uniform"), (1, 100, 300, "uniform"), (15, 10, 40, "uniform"), (16, 5, 8, "one"), (17, 5, 7, "one"),
    (33, 3, 2049, "falling"), (77, 1000, 777, "padding"), (300, 2, 100, "padding"), (1000, 1023, 64, "words"),
    (1000, 1024, 64, "words"), (1500, 300, 769, "words"), (700, 700, 520, "falling")])
def test_backward(n, rows, cols, kind, dout, table):
    announce(f"embedding gradient {n} of {rows}x{cols} {kind} {dout} {table}")
    d = (0.1 * torch.randn((n, cols), generator=torch.Generator().manual_seed(n))).to(dout).cuda()
    for width, scale in ((torch.int64, 1.0), (torch.int32, 27.5)):
        t = _tokens(n, rows, kind).to(width).cuda()
        got = pm.embedding_backward(t, d, rows, scale=scale, out_dtype=table)
        assert got.shape == (rows, cols) and got.dtype == table
        _check_backward(got, t, d, rows, scale, kind)
        assert torch.equal(got, pm.embedding_backward(t, d, rows, scale=scale, out_dtype=table))


@pytest.mark.parametrize("n", [8191, 8192, 8193, 16384, 20000, 65536, 65537])
@pytest.mark.parametrize("rows,cols,kind", [(150, 24, "words"), (40000, 9, "uniform"), (1, 8, "one"), (151936, 3, "padding")])
def test_sort_of_many_tokens(n, rows, cols, kind):
    """One workgroup's tokens and more, one pass and two, runs of 16 and of 64; equal
    tokens keep their order, so the sums are the same in every call."""
    announce(f"embedding gradient {n} of {rows}x{cols} {kind}")
    d = torch.randn((n, cols), generator=torch.Generator().manual_seed(n)).cuda()
    t = _tokens(n, rows, kind).cuda()
    got = pm.embedding_backward(t, d, rows)
    _check_backward(got, t, d, rows, 1.0, kind)
    assert torch.equal(got, pm.embedding_backward(t, d, rows))


@pytest.mark.parametrize("dout,table", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("base", [1, 9, 2041])
def test_every_row_end(base, dout, table):
    """Rows that end after each number of elements of a vector; tokens of few rows, whose
    sums go over several runs."""
    for cols in range(base, base + 8):
        announce(f"embedding gradient 90 of 4x{cols} {dout} {table}")
        t = _tokens(90, 4, "words").cuda()
        d = torch.randn((90, cols), generator=torch.Generator().manual_seed(cols)).to(dout).cuda()
        got = pm.embedding_backward(t, d, 4, out_dtype=table)
        _check_backward(got, t, d, 4, 1.0, cols)
        before = _np(got)
        pm.embedding_backward(t, d, 4, scale=-0.5, dtable=got, accumulate=True)
        _check_backward(got, t, d, 4, -0.5, cols, before)
        out = pm.embedding_forward(t, got, scale=3.0, out_dtype=dout)
        assert torch.equal(out, (got[t].float() * 3.0).to(dout))


def test_three_passes():
    """Keys of more than 20 bits."""
    announce("embedding gradient three passes")
    rows = (1 << 21) + 5
    for n in (500, 9000):
        t = _tokens(n, rows, "uniform").cuda()
        t[:4] = torch.tensor([rows - 1, 0, rows, 1 << 20])
        d = torch.randn((n, 2), device="cuda", generator=torch.Generator("cuda").manual_seed(n))
        _check_backward(pm.embedding_backward(t, d, rows), t, d, rows, 1.0, n)


@pytest.mark.parametrize("table", [F32, BF16])
def test_accumulate_pitch_and_untouched(table):
    """Windows with odd pitches and offsets, whose other elements stay; accumulate leaves
    the rows without tokens bit for bit; without it they become zero."""
    announce(f"embedding windows {table}")
    n, rows, cols = 500, 90, 101
    for kind in ("words", "padding"):
        t = _tokens(n, rows, kind).cuda()
        wide_d = torch.full((n, cols + 9), float("nan"), dtype=BF16, device="cuda")
        d = wide_d[:, 5:5 + cols]
        d.copy_(torch.randn((n, cols), generator=torch.Generator().manual_seed(2)))
        if kind == "padding":   # what padding's rows hold does not matter
            d[(t < 0) | (t >= rows)] = float("nan")
        clean = torch.nan_to_num(d)
        wide = torch.full((rows + 2, cols + 7), 2.5, dtype=table, device="cuda")
        g = wide[1:-1, 3:3 + cols]
        before = torch.randn((rows, cols), generator=torch.Generator().manual_seed(3)).to(table).cuda()
        g.copy_(before)
        assert pm.embedding_backward(t, d, rows, scale=0.5, dtable=g, accumulate=True) is g
        _check_backward(g, t, clean, rows, 0.5, "accumulate", _np(before))
        none = torch.ones(rows, dtype=torch.bool, device="cuda")
        none[t[(t >= 0) & (t < rows)]] = False
        assert torch.equal(g[none], before[none])
        pm.embedding_backward(t, d, rows, scale=0.5, dtable=g)
        _check_backward(g, t, clean, rows, 0.5, "written")
        assert (g[none] == 0).all()
        g.fill_(2.5)
        assert (wide == 2.5).all()
    weight = torch.full((12, 20), float("nan"), dtype=table, device="cuda")
    inner = weight[1:11, 4:17]
    inner.copy_(torch.randn((10, 13)))
    out = torch.full((7, 30), 4.0, device="cuda")
    o = out[1:6, 9:22]
    t = torch.tensor([3, -1, 9, 0, 10], device="cuda")
    pm.embedding_forward(t, inner, out=o)
    assert torch.equal(o[0], inner[3].float()) and torch.equal(o[2], inner[9].float()) and (o[1] == 0).all() and (o[4] == 0).all()
    o.fill_(4.0)
    assert (out == 4).all()


def test_special_values_stay_in_their_rows():
    announce("embedding special values")
    t = _tokens(400, 30, "words").cuda()
    d = torch.randn((400, 16), generator=torch.Generator().manual_seed(4)).cuda()
    want = pm.embedding_backward(t, d, 30)
    d[7, 3] = float("nan")
    d[100, 5] = float("inf")
    got = pm.embedding_backward(t, d, 30)
    assert torch.isnan(got[t[7], 3]) and torch.isinf(got[t[100], 5])
    got[t[7], 3], got[t[100], 5] = want[t[7], 3], want[t[100], 5]
    assert torch.equal(got, want)


def test_empty():
    announce("embedding empty")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.ones((4, 6), device="cuda")
    assert pm.embedding_forward(none, w).shape == (0, 6)
    g = pm.embedding_backward(none, torch.empty((0, 6), device="cuda"), 4)
    assert (g == 0).all()
    keep = torch.full((4, 6), 2.0, device="cuda")
    pm.embedding_backward(none, torch.empty((0, 6), device="cuda"), 4, dtable=keep, accumulate=True)
    assert (keep == 2).all()
    # a table without rows: every token is padding
    t = torch.tensor([0, 1], device="cuda")
    assert (pm.embedding_forward(t, torch.empty((0, 6), device="cuda")) == 0).all()
    assert pm.embedding_backward(t, torch.ones((2, 6), device="cuda"), 0).shape == (0, 6)


def test_streams_two_at_once_and_graphs():
    announce("embedding streams and graphs")
    sets = []
    for s, n in ((1, 900), (2, 9000)):
        gen = torch.Generator().manual_seed(s)
        sets.append((_tokens(n, 200, "words", s).cuda(), torch.randn((n, 136), generator=gen).bfloat16().cuda(),
                     torch.randn((200, 136), generator=gen).cuda()))

    def both(t, d, w, stream=None):
        return pm.embedding_forward(t, w, stream=stream), pm.embedding_backward(t, d, 200, stream=stream)

    want = [both(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [both(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    graphs, results = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(both(*s))
        graphs.append(graph)
    for _ in range(4):
        for r in results:
            for t in r:
                t.fill_(9.0)
        graphs[0].replay()
        both(*sets[1])
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(results, want) for a, b in zip(g, w))


def test_python_refusals():
    announce("embedding refusals")
    t = torch.tensor([1, 2, 3], device="cuda")
    w, d = torch.ones((5, 8), device="cuda"), torch.ones((3, 8), device="cuda")
    for call in (lambda: pm.embedding_forward(t.float(), w), lambda: pm.embedding_forward(t, w.half()),
                 lambda: pm.embedding_backward(t.short(), d, 5), lambda: pm.embedding_backward(t, d, 5, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: pm.embedding_forward(t[None], w), lambda: pm.embedding_forward(torch.arange(6, device="cuda")[::2], w),
                 lambda: pm.embedding_forward(t.cpu(), w), lambda: pm.embedding_forward(t, w[0]), lambda: pm.embedding_forward(t, w.t()),
                 lambda: pm.embedding_forward(t, w, out=d[:2]), lambda: pm.embedding_forward(t, w, out=d, out_dtype=torch.bfloat16),
                 lambda: pm.embedding_backward(t, d[:2], 5), lambda: pm.embedding_backward(t, d, 5, accumulate=True),
                 lambda: pm.embedding_backward(t, d, 5, dtable=torch.empty((4, 8), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pm.MuonHError):
        pm.embedding_forward(t, w, scale=float("inf"))
    with pytest.raises(pm.MuonHError):
        pm.embedding_forward(t, w, out=w[:3])
    with pytest.raises(pm.MuonHError):
        pm.embedding_backward(t, w[:3], 5, dtable=w)


def test_more_than_2_32_elements():
    """2^20 + 1 tokens of 4096 columns; the gradients are small whole numbers, whose sums
    are exact in any order."""
    n, rows, cols = (1 << 20) + 1, 300, 4096
    announce(f"embedding {n} of {rows}x{cols}")
    t = _tokens(n, rows, "padding").cuda()
    weight = torch.randn((rows, cols), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    known = (t >= 0) & (t < rows)
    at = t.clamp(0, rows - 1)
    out = pm.embedding_forward(t, weight)
    for s in range(0, n, 1 << 17):
        part = slice(s, s + (1 << 17))
        assert torch.equal(out[part], torch.where(known[part, None], weight[at[part]], torch.zeros_like(weight[:1])))
    out.random_(-2, 3)
    got = pm.embedding_backward(t, out, rows)
    for s in range(0, cols, 512):
        d = torch.where(known[:, None], out[:, s:s + 512], torch.zeros_like(out[:1, :1])).float()
        assert torch.equal(got[:, s:s + 512], torch.zeros((rows, 512), device="cuda").index_add_(0, at, d))
    del out, d
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,rows", [(n, r) for n, r, _, _, path in SORTS if path != "ranked" and r < 1 << 30])
def test_sorts_of_every_plan(n, rows):
    """One, two and three passes over few and over more than 32 workgroups, skewed tokens
    and padding; the sizes' plans are pinned on the host."""
    for kind, cols in (("words", 2), ("padding", 3), ("one", 1)):
        announce(f"embedding gradient {n} of {rows}x{cols} {kind}")
        t = _tokens(n, rows, kind).cuda()
        t[:5] = torch.tensor([rows - 1, 0, rows, -1, rows // 2])
        d = torch.randn((n, cols), generator=torch.Generator().manual_seed(n)).cuda()
        got = pm.embedding_backward(t, d, rows)
        _check_backward(got, t, d, rows, 1.0, kind)
        assert torch.equal(got, pm.embedding_backward(t, d, rows))


@pytest.mark.parametrize("n,rows", [(n, r) for n, r, _, _, path in SORTS if r == 1 << 30])
def test_four_passes(n, rows):
    """The most rows: keys of 31 bits.  Small whole numbers, whose sums are exact."""
    announce(f"embedding gradient {n} of {rows}x1")
    gen = torch.Generator("cuda").manual_seed(n)
    t = torch.randint(0, rows, (n,), device="cuda", generator=gen)
    t[::5] = t[3::5][torch.randint(0, 50, (len(t[::5]),), device="cuda", generator=gen)]
    t[:5] = torch.tensor([rows - 1, 0, rows, -1, 1 << 20])
    d = torch.randint(1, 3, (n, 1), device="cuda", generator=gen).float()
    got = pm.embedding_backward(t, d, rows)
    known = (t >= 0) & (t < rows)
    row, where = torch.unique(t[known], return_inverse=True)
    want = torch.zeros(len(row), device="cuda").index_add_(0, where, d[known, 0])
    assert torch.equal(got[row, 0], want) and int((got != 0).sum()) == len(row)
    del got
    torch.cuda.empty_cache()
