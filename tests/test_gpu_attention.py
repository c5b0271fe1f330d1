"""Causal attention over packed sequences and its gradients, on an MI355X against
the fp64 oracle.

Tolerances, element by element (u = 2^-23: fp32 sums whose additions may truncate;
b = 2^-8: half a step of bf16).  With n rows seen and D columns:
  S:    es_ij = c D u sum|q k|
  P:    the exponent's product, difference and 2^x: ep_ij = es_ij + 8 u (|S_ij| + |lse_i| + 1),
        and b for the matrix operand
  out:  sum_j P |v| (b + 2 max_j ep_ij + 2 n u), and b (the maximum over j: numerator
        and denominator)
  lse:  max_j ep_ij + n u
  dP:   D u sum|do v|;  delta: D u sum|do o|;  together ed_ij
  dS:   eds_ij = |dS| (b + 2 ep_ij) + c P (ed_ij + 2 u |dP - delta|)
  dq:   sum_j (eds |k| + 2 n u |dS k|), and b;  dk likewise over the rows and heads
  dv:   sum_i P |do| (b + 2 ep + 2 n u), and b
In the backward pass out and lse are inputs, the same for both sides.
"""

import ctypes

import numpy as np
import pytest
import torch

import pretraining_optimizer_amd as pm
from pretraining_optimizer_amd import muonh as mb
from oracle import attention
from parity import announce

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -23, 2.0 ** -8


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(lens, heads, kv, dim, seed=0, tail=0, spread=1.5):
    gen = torch.Generator().manual_seed(seed + 7 * sum(lens) + dim)
    n = sum(lens) + tail
    q = (spread * torch.randn((n, heads, dim), generator=gen)).bfloat16()
    k, v, do = (torch.randn((n, h, dim), generator=gen).bfloat16() for h in (kv, kv, heads))
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    return q.cuda(), k.cuda(), v.cuda(), (0.1 * do).bfloat16().cuda(), cu.cuda()


def _each(q, k, v, cu, scale):
    """Per sequence and head: rows, head, key head, |S|, lse, P and the error of S."""
    Q, K, V = _np(q), _np(k), _np(v)
    tokens, heads, dim = Q.shape
    group = heads // K.shape[1]
    ends = [min(max(int(c), 0), tokens) for c in cu.tolist()]
    for s, e in zip(ends[:-1], ends[1:]):
        for h in range(heads if e > s else 0):
            rows, g = slice(s, e), h // group
            a, b = Q[rows, h], K[rows, g]
            S, lse, P = attention.probabilities(a, b, scale)
            low = P > 0
            S = np.where(low, np.abs(np.where(low, S, 0.0)), 0.0)
            es = np.where(low, scale * dim * U * (np.abs(a) @ np.abs(b).T), 0.0)
            ep = np.where(low, es + 8 * U * (S + np.abs(lse)[:, None] + 1), 0.0)
            yield rows, h, g, a, b, V[rows, g], lse, P, ep


def _check_forward(out, lse, q, k, v, cu, scale, what):
    O, L = _np(out), _np(lse)
    for rows, h, g, a, b, vh, rl, P, ep in _each(q, k, v, cu, scale):
        n, worst = len(a), ep.max(axis=1)
        want = P @ vh
        tol = (P @ np.abs(vh)) * (B + 2 * worst + 2 * n * U)[:, None]
        tol += B * (np.abs(want) + tol)
        err = np.abs(O[rows, h] - want)
        assert np.all(err <= tol), (what, "out", rows, h, float((err - tol).max()))
        err = np.abs(L[h, rows] - rl)
        assert np.all(err <= worst + n * U), (what, "lse", rows, h, float(err.max()))


def _check_backward(grads, do, q, k, v, out, lse, cu, scale, what):
    dQ, dK, dV = (_np(t) for t in grads)
    DO, O, L = _np(do), _np(out), _np(lse)
    rdq, rdk, rdv = attention.attention_backward(DO, _np(q), _np(k), _np(v), O, L, cu.tolist(), scale)
    tq, tk, tv = (np.zeros(t.shape) for t in (rdq, rdk, rdv))
    dim, group = q.shape[2], q.shape[1] // k.shape[1]
    for rows, h, g, a, b, vh, rl, P, ep in _each(q, k, v, cu, scale):
        n, d = len(a), DO[rows, h]
        # the given lse is the formula's: P's error from it is the reference's, too
        P = P * np.exp(rl - L[h, rows])[:, None]
        dP = d @ vh.T
        delta = (d * O[rows, h]).sum(axis=1, keepdims=True)
        ed = dim * U * (np.abs(d) @ np.abs(vh).T + np.abs(d * O[rows, h]).sum(axis=1, keepdims=True))
        ds = scale * P * (dP - delta)
        eds = np.abs(ds) * (B + 2 * ep) + scale * P * (ed + 2 * U * np.abs(dP - delta))
        m = group * n
        tq[rows, h] = eds @ np.abs(b) + 2 * n * U * (np.abs(ds) @ np.abs(b))
        tk[rows, g] += eds.T @ np.abs(a) + 2 * m * U * (np.abs(ds).T @ np.abs(a))
        tv[rows, g] += (P * (B + 2 * ep + 2 * m * U)).T @ np.abs(d)
    for name, got, want, tol in (("dq", dQ, rdq, tq), ("dk", dK, rdk, tk), ("dv", dV, rdv, tv)):
        live = np.isfinite(want)
        tol = tol + B * (np.abs(want) + tol)
        err = np.abs(got - want)
        assert np.all(err[live] <= tol[live]), (what, name, float((err - tol)[live].max()))


def _both(q, k, v, do, cu, scale, what):
    out, lse = pm.attention_forward(q, k, v, cu, scale=scale)
    real = q.shape[2] ** -0.5 if scale is None else scale
    _check_forward(out, lse, q, k, v, cu, real, what)
    grads = pm.attention_backward(do, q, k, v, out, lse, cu, scale=scale)
    _check_backward(grads, do, q, k, v, out, lse, cu, real, what)
    again = pm.attention_backward(do, q, k, v, out, lse, cu, scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    out2, lse2 = pm.attention_forward(q, k, v, cu, scale=scale)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    return out, lse, grads


LENS = [[1], [2], [31], [32], [33], [63, 65], [64], [77], [127], [128], [129], [1, 1, 1], [200, 1, 0, 300], [0, 5, 0],
        [257, 63], [500]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "+".join(map(str, v)))
@pytest.mark.parametrize("heads,kv,dim", [(4, 2, 128), (3, 1, 64)])
def test_lengths(lens, heads, kv, dim):
    announce(f"attention {lens} {heads}/{kv} heads of {dim}")
    _both(*_inputs(lens, heads, kv, dim), None, f"{lens}")


def _heads_for_large_blocks(lens):
    """The least heads whose blocks of 128 rows are a workgroup per CU, so that neither
    the rows' nor the keys' kernels take smaller ones."""
    return -(-256 // (sum(lens) // 128 + len(lens)))


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "+".join(map(str, v)))
@pytest.mark.parametrize("group,dim", [(1, 128), (2, 64)])
def test_lengths_in_large_blocks(lens, group, dim):
    kv = _heads_for_large_blocks(lens)
    announce(f"attention {lens} {group * kv}/{kv} heads of {dim}")
    _both(*_inputs(lens, group * kv, kv, dim), None, f"{lens}")


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "+".join(map(str, v)))
@pytest.mark.parametrize("group,dim", [(1, 128), (2, 64)])
def test_lengths_in_blocks_between(lens, group, dim):
    """More workgroups of 128 rows than half the CUs, and fewer than all of them."""
    kv = -(-140 // (group * (sum(lens) // 128 + len(lens))))
    announce(f"attention {lens} {group * kv}/{kv} heads of {dim}")
    _both(*_inputs(lens, group * kv, kv, dim), None, f"{lens}")


@pytest.mark.parametrize("dim", [8, 40, 72, 104])
def test_head_widths_in_large_blocks(dim):
    announce(f"attention width {dim}, large blocks")
    _both(*_inputs([150, 70], 86, 86, dim), 0.2, f"dim {dim}")


def test_rows_in_large_blocks_and_keys_in_small_ones():
    """Many heads that read few key heads."""
    announce("attention 64/2 heads")
    _both(*_inputs([530, 260], 64, 2, 64), None, "64/2")


def test_more_than_64_sequences():
    """Their blocks keep the sequences' order; empty ones and single tokens among them."""
    announce("attention 65 and 200 sequences")
    _both(*_inputs([37 * i % 131 for i in range(65)], 2, 1, 64), None, "65 sequences")
    _both(*_inputs([i * i % 17 for i in range(200)], 4, 2, 64), None, "200 sequences")
    _both(*_inputs([0] * 70 + [300] + [0] * 70 + [1], 4, 4, 128), None, "142 sequences")


def test_offsets_beyond_32_bits():
    """Tokens 2^22 elements apart: the last lie beyond 2^31 elements, and 2^32 bytes."""
    announce("attention large pitch")
    lens, heads, kv, dim = [300, 250], 2, 1, 64
    q, k, v, do, cu = _inputs(lens, heads, kv, dim)
    want = pm.attention_forward(q, k, v, cu)
    wantg = pm.attention_backward(do, q, k, v, *want, cu)
    wide = torch.empty((sum(lens), 1 << 22), dtype=torch.bfloat16, device="cuda")
    at = 0
    views = []
    for t in (q, k, v, do, want[0], q, k, v):
        n = t.shape[1] * dim
        views.append(wide[:, at:at + n].unflatten(1, (-1, dim)))
        views[-1].copy_(t)
        at += n
    fq, fk, fv, fdo, fo, gq, gk, gv = views
    out, lse = pm.attention_forward(fq, fk, fv, cu, out=fo)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    pm.attention_backward(fdo, fq, fk, fv, out, lse, cu, dq=gq, dk=gk, dv=gv)
    assert all(torch.equal(a, b) for a, b in zip((gq, gk, gv), wantg))
    del wide, views
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 56, 64, 72, 80, 96, 104, 120, 128])
def test_head_widths(dim):
    announce(f"attention width {dim}")
    _both(*_inputs([150, 70], 4, 2, dim), 0.2, f"dim {dim}")


@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 8), (8, 1), (6, 3), (5, 5), (16, 2)])
def test_groups(heads, kv):
    announce(f"attention {heads}/{kv} heads")
    _both(*_inputs([170, 90], heads, kv, 64), None, f"{heads}/{kv}")


def test_longer_sequences():
    """Many tiles per row, in small and in large blocks."""
    announce("attention 1500+700, 64 sequences")
    _both(*_inputs([1500, 700], 2, 1, 128), None, "1500+700")
    _both(*_inputs([1000, 777], 12, 12, 64), None, "1000+777")
    _both(*_inputs([1100, 700], 16, 16, 128), None, "1100+700")
    _both(*_inputs([13 * i % 97 for i in range(64)], 2, 2, 64), None, "64 sequences")


@pytest.mark.parametrize("dim,kv", [(64, 1), (128, 2), (40, 2)])
def test_a_long_sequence(dim, kv):
    """One sequence of 20011 tokens: some of its rows and keys, to the module's
    tolerances; keys are summed over the heads of a group."""
    n, heads = 20011, 2
    announce(f"attention {n} tokens, 2/{kv} heads of {dim}")
    q, k, v, do, cu = _inputs([n], heads, kv, dim)
    out, lse = pm.attention_forward(q, k, v, cu)
    grads = pm.attention_backward(do, q, k, v, out, lse, cu)
    Q, K, V, DO, O, L = (_np(t) for t in (q, k, v, do, out, lse))
    dQ, dK, dV = (_np(t) for t in grads)
    c, group = dim ** -0.5, heads // kv
    at = [0, 1, 31, 32, 127, 128, 8191, 10000, n - 129, n - 2, n - 1]

    def close(got, want, tol, what):
        tol = tol + B * (np.abs(want) + tol)
        assert np.all(np.abs(got - want) <= tol), (what, float((np.abs(got - want) - tol).max()))

    delta = (DO * O).sum(axis=2)          # [tokens, heads]
    size = np.abs(DO * O).sum(axis=2)
    for i in at:
        for h in range(heads):
            g, m = h // group, i + 1
            S = c * (K[:m, g] @ Q[i, h])
            ep = c * dim * U * (np.abs(K[:m, g]) @ np.abs(Q[i, h])) + 8 * U * (np.abs(S) + abs(L[h, i]) + 1)
            top = S.max()
            rl = top + np.log(np.exp(S - top).sum())
            P = np.exp(S - rl)
            assert abs(L[h, i] - rl) <= ep.max() + m * U, ("lse", i, h)
            close(O[i, h], P @ V[:m, g], (P @ np.abs(V[:m, g])) * (B + 2 * ep.max() + 2 * m * U), ("out", i, h))
            P = np.exp(S - L[h, i])
            dP = V[:m, g] @ DO[i, h]
            ed = dim * U * (np.abs(V[:m, g]) @ np.abs(DO[i, h]) + size[i, h])
            ds = c * P * (dP - delta[i, h])
            eds = np.abs(ds) * (B + 2 * ep) + c * P * (ed + 2 * U * np.abs(dP - delta[i, h]))
            close(dQ[i, h], ds @ K[:m, g], eds @ np.abs(K[:m, g]) + 2 * m * U * (np.abs(ds) @ np.abs(K[:m, g])), ("dq", i, h))
    for j in at:
        for g in range(kv):
            wk = wv = tk = tv = 0.0
            for h in range(g * group, (g + 1) * group):
                a, d, m = Q[j:, h], DO[j:, h], group * (n - j)
                S = c * (a @ K[j, g])
                ep = c * dim * U * (np.abs(a) @ np.abs(K[j, g])) + 8 * U * (np.abs(S) + np.abs(L[h, j:]) + 1)
                P = np.exp(S - L[h, j:])
                dP = d @ V[j, g]
                ed = dim * U * (np.abs(d) @ np.abs(V[j, g]) + size[j:, h])
                ds = c * P * (dP - delta[j:, h])
                eds = np.abs(ds) * (B + 2 * ep) + c * P * (ed + 2 * U * np.abs(dP - delta[j:, h]))
                wk, wv = wk + ds @ a, wv + P @ d
                tk = tk + eds @ np.abs(a) + 2 * m * U * (np.abs(ds) @ np.abs(a))
                tv = tv + (P * (B + 2 * ep + 2 * m * U)) @ np.abs(d)
            close(dK[j, g], wk, tk, ("dk", j, g))
            close(dV[j, g], wv, tv, ("dv", j, g))


@pytest.mark.parametrize("dim", [64, 128])
def test_peaked_and_growing_scores(dim):
    """Scores far apart, and maxima that grow along a row by more and by less than the
    factor from which the output is rescaled."""
    announce(f"attention peaked {dim}")
    q, k, v, do, cu = _inputs([300, 40], 2, 1, dim, seed=3)
    _both(q * 8, k, v, do, cu, None, "peaked")
    ramp = torch.linspace(0.1, 6.0, len(k), device="cuda")[:, None, None]
    _both(q.abs(), (k.abs() * ramp).bfloat16(), v, do, cu, None, "growing")
    _both(q.abs(), (k.abs() * ramp.flip(0)).bfloat16(), v, do, cu, None, "falling")
    _both(q.abs(), (-k.abs() * 20).bfloat16(), v, do, cu, None, "far below zero")
    zero = torch.zeros_like(q)
    _both(zero, k, v, do, cu, 3.0, "equal scores")


def _windows(tokens, heads, kv, dim, pad=8):
    """q, k, v as slices of one fused matrix with other columns behind."""
    wide = torch.full((tokens, (heads + 2 * kv) * dim + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    parts = wide[:, :heads * dim], wide[:, heads * dim:(heads + kv) * dim], wide[:, (heads + kv) * dim:(heads + 2 * kv) * dim]
    return wide, [p.unflatten(1, (-1, dim)) for p in parts]


@pytest.mark.parametrize("dim", [40, 64, 128])
def test_fused_buffers_and_tokens_behind_the_last_sequence(dim):
    """Slices of a fused projection and of a fused gradient; rows that no sequence
    holds are NaN in the inputs and stay as they were in the results."""
    announce(f"attention windows {dim}")
    heads, kv, lens, tail = 4, 2, [130, 35], 70
    q, k, v, do, cu = _inputs(lens, heads, kv, dim, tail=tail)
    n, live = len(q), sum(lens)
    want_out, want_lse = pm.attention_forward(q[:live], k[:live], v[:live], cu)
    want = pm.attention_backward(do[:live], q[:live], k[:live], v[:live], want_out, want_lse, cu)
    fused, (fq, fk, fv) = _windows(n, heads, kv, dim)
    for a, b in ((fq, q), (fk, k), (fv, v)):
        a.copy_(b)
        a[live:] = float("nan")
    out = torch.full((n, heads * dim + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    o = out[:, 8:8 + heads * dim].unflatten(1, (heads, dim))
    lse = torch.full((heads, n), 3.0, device="cuda")
    got = pm.attention_forward(fq, fk, fv, cu, out=o, lse=lse)
    assert got[0] is o and got[1] is lse
    assert torch.equal(o[:live], want_out) and torch.equal(lse[:, :live], want_lse)
    assert (out[live:] == 3).all() and (out[:, :8] == 3).all() and (out[:, 8 + heads * dim:] == 3).all()
    assert (lse[:, live:] == 3).all()
    do = do.clone()
    do[live:] = float("nan")
    lse[:, live:] = float("nan")
    o[live:] = float("nan")
    grads, (gq, gk, gv) = _windows(n, heads, kv, dim)
    pm.attention_backward(do, fq, fk, fv, o, lse, cu, dq=gq, dk=gk, dv=gv)
    for a, b in zip((gq, gk, gv), want):
        assert torch.equal(a[:live], b)
    assert (grads[live:] == 7).all() and (grads[:, -8:] == 7).all()
    assert (fused[:, -8:] == 7).all()


@pytest.mark.parametrize("dim,kv", [(64, 1), (128, 1), (64, 64), (64, 20)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", [0, 5, 31, 32, 40, 63, 64, 100, 149])
def test_special_values_reach_later_rows_only(where, value, dim, kv):
    """An Inf or NaN in a token's key or value: other sequences keep their results bit
    for bit, earlier rows and other columns theirs (within the tolerances: a block
    with such a value adds its keys one at a time), and the rest is what the formula
    gives."""
    announce(f"attention {value} at {where}, width {dim}, {kv} key heads")
    q, k, v, do, cu = _inputs([20, 150, 30], 2 * kv, kv, dim)
    want, wl = pm.attention_forward(q, k, v, cu)
    later = slice(20 + where, 170)
    for t in (k, v):
        bad = t.clone()
        bad[20 + where, :, 3] = value
        out, lse = pm.attention_forward(q, bad if t is k else k, bad if t is v else v, cu)
        for s in (slice(0, 20), slice(170, 200)):
            assert torch.equal(out[s], want[s]) and torch.equal(lse[:, s], wl[:, s])
        hit, hit_lse = out[later].clone(), lse[:, later].clone()
        if t is v:
            # every row that sees it has P > 0
            assert torch.equal(lse, wl)
            assert (torch.isnan(hit[:, :, 3]).all() if value != value else (hit[:, :, 3] == value).all())
            out[later, :, 3] = want[later, :, 3]
        else:
            if value != value:
                assert torch.isnan(hit).all() and torch.isnan(hit_lse).all()
            out[later], lse[:, later] = want[later], wl[:, later]
        _check_forward(out, lse, q, k, v, cu, dim ** -0.5, f"{value} at {where}")


@pytest.mark.parametrize("kv", [1, 20, 32])
def test_scores_of_minus_infinity(kv):
    """Keys whose scores are -inf for every row: rows that see others as well have what
    the formula gives, in a wavefront that sees only such keys, too."""
    announce(f"attention minus infinity, {kv} key heads")
    q, k, v, do, cu = _inputs([200, 90], 2 * kv, kv, 64)
    q = q.abs() + 0.5
    k[:96, :, 5] = -float("inf")
    out, lse = pm.attention_forward(q, k, v, cu)
    # a row without a finite score is no number
    assert torch.isnan(out[:96]).all()
    kept, at = torch.cat([k[96:200], k[200:]]), torch.tensor([0, 104, 194], dtype=torch.int32, device="cuda")
    _check_forward(out[96:], lse[:, 96:], q[96:], kept, v[96:], at, 64 ** -0.5, "minus infinity")


def test_gradients_of_other_sequences_are_kept():
    announce("attention backward NaN in one sequence")
    q, k, v, do, cu = _inputs([70, 90, 50], 2, 1, 64)
    out, lse = pm.attention_forward(q, k, v, cu)
    want = pm.attention_backward(do, q, k, v, out, lse, cu)
    for i in range(6):
        args = [t.clone() for t in (do, q, k, v, out, lse)]
        if i == 5:
            args[5][:, 70:160] = float("nan")
        else:
            args[i][70:160] = float("nan")
        got = pm.attention_backward(*args, cu)
        for a, b in zip(got, want):
            assert torch.equal(a[:70], b[:70]) and torch.equal(a[160:], b[160:])


def test_ends_outside_the_tokens():
    """The device's cu_seqlens is taken into the tokens; a sequence that would end before
    it starts is empty."""
    announce("attention ends outside")
    q, k, v, do, _ = _inputs([200], 2, 1, 64)
    for raw, clean in (([-5, 70, 1 << 30], [0, 70, 200]), ([10, 60, 60, 150], [10, 60, 150]),
                       ([300, 400], None), ([90, 40], None)):
        cu = torch.tensor(raw, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 3.0), torch.full((2, 200), 3.0, device="cuda")
        pm.attention_forward(q, k, v, cu, out=out, lse=lse)
        grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
        pm.attention_backward(do, q, k, v, out, lse, cu, dq=grads[0], dk=grads[1], dv=grads[2])
        if clean is None:
            assert all((t == 3).all() for t in [out, lse] + grads)
            continue
        _check_forward(out, lse, q, k, v, torch.tensor(clean), 64 ** -0.5, raw)
        _check_backward(grads, do, q, k, v, out, lse, torch.tensor(clean), 64 ** -0.5, raw)
        for s in (slice(0, clean[0]), slice(clean[-1], 200)):
            assert (out[s] == 3).all() and all((t[s] == 3).all() for t in grads)


def test_empty():
    announce("attention empty")
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = pm.attention_forward(q, q, q, cu)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert [t.shape for t in pm.attention_backward(q, q, q, q, out, lse, cu)] == [(0, 4, 64)] * 3
    # no sequences at all: nothing is written
    x = torch.ones((5, 2, 8), dtype=torch.bfloat16, device="cuda")
    one = cu[:1].clone()
    out, lse = pm.attention_forward(x, x, x, one, out=torch.full_like(x, 2.0))
    assert (out == 2).all()
    grads = pm.attention_backward(x, x, x, x, out, lse, one, dq=torch.full_like(x, 5.0))
    assert (grads[0] == 5).all()


def test_streams_two_at_once_and_graphs():
    """Two calls on streams of their own, and two graphs of the whole pass replayed in
    turn with eager work between, each against the eager result."""
    announce("attention streams and graphs")
    sets = [_inputs([300, 57], 4, 2, 64, seed=s) for s in (1, 2)]
    want = []
    for q, k, v, do, cu in sets:
        out, lse = pm.attention_forward(q, k, v, cu)
        want.append((out, lse) + pm.attention_backward(do, q, k, v, out, lse, cu))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (q, k, v, do, cu), st in zip(sets, streams):
            out, lse = pm.attention_forward(q, k, v, cu, stream=st)
            got.append((out, lse) + pm.attention_backward(do, q, k, v, out, lse, cu, stream=st))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    graphs, results = [], []
    for q, k, v, do, cu in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse = pm.attention_forward(q, k, v, cu)
            results.append((out, lse) + pm.attention_backward(do, q, k, v, out, lse, cu))
        graphs.append(graph)
    for _ in range(4):
        for t in results[0] + results[1]:
            t.fill_(9.0)
        graphs[0].replay()
        with torch.cuda.stream(streams[0]):
            pm.attention_forward(*sets[1][:3], sets[1][4])
        graphs[1].replay()
        torch.cuda.synchronize()
        for g, w in zip(results, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_python_refusals():
    announce("attention refusals")
    q, k, v, do, cu = _inputs([40], 4, 2, 64)
    out, lse = pm.attention_forward(q, k, v, cu)
    with pytest.raises(TypeError):
        pm.attention_forward(q.float(), k, v, cu)
    with pytest.raises(TypeError):
        pm.attention_forward(q, k.half(), v, cu)
    with pytest.raises(ValueError):
        pm.attention_forward(q, k, v[:, :1], cu)
    with pytest.raises(ValueError):
        pm.attention_forward(q, k, v[:30], cu)
    with pytest.raises(ValueError):
        pm.attention_forward(q[0], k, v, cu)
    with pytest.raises(ValueError):
        pm.attention_forward(q, k, v, cu.long())
    with pytest.raises(ValueError):
        pm.attention_forward(q, k, v, cu[:0])
    with pytest.raises(ValueError):
        pm.attention_forward(q, k, v, cu.cpu())
    with pytest.raises(ValueError):
        pm.attention_forward(q[:, ::2], k, v, cu)
    with pytest.raises(ValueError):
        pm.attention_forward(q, k, v, cu, lse=lse[:2])
    with pytest.raises(pm.MuonHError):
        pm.attention_forward(q, k, v, cu, scale=0.0)
    with pytest.raises(pm.MuonHError):
        pm.attention_forward(q, k, v, cu, scale=float("nan"))
    with pytest.raises(pm.MuonHError):
        pm.attention_forward(q, k, v, cu, out=q)
    with pytest.raises(pm.MuonHError):
        pm.attention_forward(q[:, :3].contiguous(), k, v, cu)
    odd = torch.zeros((40, 4 * 64 + 1), dtype=torch.bfloat16, device="cuda")[:, 1:].unflatten(1, (4, 64))
    with pytest.raises(pm.MuonHError):
        pm.attention_forward(odd, k, v, cu)
    with pytest.raises(ValueError):
        pm.attention_backward(do, q, k, v, None, lse, cu)
    with pytest.raises(ValueError):
        pm.attention_backward(do[:, :2], q, k, v, out, lse, cu)
    with pytest.raises(pm.MuonHError):
        pm.attention_backward(do, q, k, v, out, lse, cu, dq=do)
    wide = torch.empty((1, 4, 136), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pm.MuonHError):
        pm.attention_forward(wide, wide, wide, cu)


def _seen_softmax(q, k, v, scale, seen):
    """out, lse and their tolerances of one head, for rows that see the keys of `seen`
    [rows, keys]; NaN for a row that sees none."""
    n, dim = q.shape
    S = np.where(seen, scale * (q @ k.T), -np.inf)
    top = S.max(axis=1)
    some = np.isfinite(top)
    top = np.where(some, top, 0.0)
    lse = np.where(some, top + np.log(np.maximum(np.exp(S - top[:, None]).sum(axis=1), 1e-300)), np.nan)
    P = np.exp(S - np.where(some, lse, 0.0)[:, None])
    size = np.where(seen, np.abs(np.where(seen, S, 0.0)) + np.abs(lse)[:, None] + 1, 0.0)
    worst = np.where(seen, scale * dim * U * (np.abs(q) @ np.abs(k).T) + 8 * U * size, 0.0).max(axis=1)
    out = np.where(some[:, None], P @ v, np.nan)
    tol = (P @ np.abs(v)) * (B + 2 * worst + 2 * n * U)[:, None]
    return out, lse, tol + B * (np.abs(out) + tol), worst + n * U


# heads of one sequence of 300 tokens: rows in four parts, in two, in one; of 64 columns and of 128
SPLITS = [(2, 64), (2, 128), (30, 64), (30, 128), (90, 64)]


@pytest.mark.parametrize("heads,dim", SPLITS)
@pytest.mark.parametrize("masked", [32, 64, 70, 128, 200])
def test_keys_that_only_some_rows_of_a_wavefront_see(masked, heads, dim):
    """The first keys hold bf16's lowest value in a spare column, where some rows' q has 8
    and the others' 0: those rows' scores are -inf there, beside rows whose scores are finite.
    A row has what the formula gives without its masked keys; where it sees no other, lse
    is -inf, the logarithm of an empty sum, and out NaN."""
    announce(f"attention {masked} keys masked for some rows, {heads} heads of {dim}")
    n = 300
    q, k, v, do, cu = _inputs([n], heads, heads, dim)
    flagged = torch.arange(n, device="cuda") * 7 % 16 < 9
    q[:, :, -1] = torch.where(flagged, 8.0, 0.0).bfloat16()[:, None]
    k[:, :, -1] = 0.0
    k[:masked, :, -1] = torch.finfo(torch.bfloat16).min
    out, lse = pm.attention_forward(q, k, v, cu)
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    seen = (j <= i) & ~(_np(flagged.float())[:, None].astype(bool) & (j < masked))
    clean = _np(k)
    clean[:, :, -1] = 0.0   # masked keys are left out by `seen`, elsewhere q or k is 0 there
    O, L, Q, V = _np(out), _np(lse), _np(q), _np(v)
    assert np.array_equal(L == -np.inf, np.broadcast_to(~seen.any(axis=1), L.shape)) and not np.isnan(L).any()
    for h in {0, heads // 2, heads - 1}:
        want, wl, tol, ltol = _seen_softmax(Q[:, h], clean[:, h], V[:, h], dim ** -0.5, seen)
        some = seen.any(axis=1)
        assert np.all(np.abs(O[some, h] - want[some]) <= tol[some]), (h, "out")
        assert np.isnan(O[~some, h]).all()
        assert np.all(np.abs(L[h, some] - wl[some]) <= ltol[some]), (h, "lse")


@pytest.mark.parametrize("heads,dim", SPLITS)
def test_gradients_of_keys_that_only_some_rows_see(heads, dim):
    """As above, with rows masked only where they see other keys, so that all have a
    result: masked keys add nothing to the gradients of those rows, nor these to theirs."""
    announce(f"attention gradients of masked keys, {heads} heads of {dim}")
    n, masked = 300, 100
    q, k, v, do, cu = _inputs([n], heads, heads, dim)
    at = torch.arange(n, device="cuda")
    flagged = (at * 7 % 16 < 9) & (at >= masked)
    q[:, :, -1] = torch.where(flagged, 8.0, 0.0).bfloat16()[:, None]
    k[:, :, -1] = 0.0
    clean = k.clone()
    k[:masked, :, -1] = torch.finfo(torch.bfloat16).min
    out, lse = pm.attention_forward(q, k, v, cu)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    dq, dk, dv = (_np(t) for t in pm.attention_backward(do, q, k, v, out, lse, cu))
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    seen = (j <= i) & ~(_np(flagged.float())[:, None].astype(bool) & (j < masked))
    Q, K, V, DO, O, L = (_np(t) for t in (q, clean, v, do, out, lse))
    c = dim ** -0.5
    for h in {0, heads // 2, heads - 1}:
        a, b, vh, d = Q[:, h], K[:, h], V[:, h], DO[:, h]
        S = c * (a @ b.T)
        P = np.where(seen, np.exp(np.where(seen, S, 0.0) - L[h][:, None]), 0.0)
        ep = c * dim * U * (np.abs(a) @ np.abs(b).T) + 8 * U * (np.abs(S) + np.abs(L[h])[:, None] + 1)
        delta = (d * O[:, h]).sum(axis=1, keepdims=True)
        ed = dim * U * (np.abs(d) @ np.abs(vh).T + np.abs(d * O[:, h]).sum(axis=1, keepdims=True))
        dP = d @ vh.T
        ds = c * P * (dP - delta)
        eds = np.abs(ds) * (B + 2 * ep) + c * P * (ed + 2 * U * np.abs(dP - delta))
        for name, got, want, tol in (
                # the spare column of dq is a sum of products with the lowest value
                ("dq", dq[:, h, :-1], (ds @ b)[:, :-1], (eds @ np.abs(b) + 2 * n * U * (np.abs(ds) @ np.abs(b)))[:, :-1]),
                ("dk", dk[:, h], ds.T @ a, eds.T @ np.abs(a) + 2 * n * U * (np.abs(ds).T @ np.abs(a))),
                ("dv", dv[:, h], P.T @ d, (P * (B + 2 * ep + 2 * n * U)).T @ np.abs(d))):
            tol = tol + B * (np.abs(want) + tol)
            assert np.all(np.abs(got - want) <= tol), (name, h, float((np.abs(got - want) - tol).max()))


def _fill_free_memory(*shapes):
    """Leaves NaN in memory that the next tensors of these shapes and types are given."""
    held = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("lens,front,tail", [
    ([130, 35], 0, 70), ([130, 35], 9, 0), ([77], 0, 1), ([77], 300, 500), ([0], 0, 5), ([], 3, 4), ([128], 0, 128),
    ([3] * 64, 1, 100), ([3] * 65, 1, 100), ([40, 0] * 40 + [0] * 20, 200, 300)], ids=str)
@pytest.mark.parametrize("heads,kv,dim", [(2, 1, 64), (4, 2, 40), (2, 2, 128), (90, 90, 64), (32, 16, 128)])
def test_new_results_are_zero_where_no_sequence_is(lens, front, tail, heads, kv, dim):
    """Padded batches: results that the call makes are zeros in the rows before the first
    sequence and behind the last one; the others' are those of the sequences alone."""
    announce(f"attention {len(lens)} sequences of {sum(lens)}, {front} rows before and {tail} behind, {heads}/{kv} heads of {dim}")
    bf16 = torch.bfloat16
    n, live = front + sum(lens) + tail, slice(front, front + sum(lens))
    q, k, v, do, _ = _inputs([n], heads, kv, dim)
    cu = torch.tensor([front] + list(front + np.cumsum(lens)), dtype=torch.int32, device="cuda")
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[live] = False
    for t in (q, k, v, do):
        t[rest] = float("nan")
    qs, ks, rows = ((n, heads, dim), bf16), ((n, kv, dim), bf16), ((heads, n), torch.float32)
    held = [torch.full(s, 3.0, dtype=t, device="cuda") for s, t in (qs, rows, qs, ks, ks)]
    pm.attention_forward(q, k, v, cu, out=held[0], lse=held[1])
    pm.attention_backward(do, q, k, v, held[0], held[1], cu, dq=held[2], dk=held[3], dv=held[4])
    assert all((t[rest] == 3).all() for t in (held[0], *held[2:])) and (held[1][:, rest] == 3).all()
    _fill_free_memory(qs, rows)
    out, lse = pm.attention_forward(q, k, v, cu)
    _fill_free_memory(qs, ks, ks)
    grads = pm.attention_backward(do, q, k, v, out, lse, cu)
    for got, kept in zip((out, lse.T, *grads), (held[0], held[1].T, *held[2:])):
        assert torch.equal(got[live], kept[live])
        assert (got[rest] == 0).all()
    # a part of the results given
    _fill_free_memory(qs, rows)
    mine = torch.full_like(q, 3.0)
    _, lse = pm.attention_forward(q, k, v, cu, out=mine)
    assert torch.equal(mine, held[0]) and (lse[:, rest] == 0).all()
    _fill_free_memory(qs, ks)
    mine = torch.full_like(k, 3.0)
    dq, dk, dv = pm.attention_backward(do, q, k, v, out, lse, cu, dv=mine)
    assert torch.equal(mine, held[4]) and (dq[rest] == 0).all() and (dk[rest] == 0).all()


def test_a_captured_call_whose_sequences_change():
    """cu_seqlens is read by the device, so a graph's sequences may become shorter: rows
    that they leave are zeros in the graph's results, on a stream of its own, too."""
    announce("attention graph with changing sequences")
    q, k, v, do, _ = _inputs([300], 4, 2, 64)
    cu = torch.tensor([0, 180, 300], dtype=torch.int32, device="cuda")
    both = lambda st=None: (lambda r: r + pm.attention_backward(do, q, k, v, *r, cu, stream=st))(  # noqa: E731
        pm.attention_forward(q, k, v, cu, stream=st))
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = both()
    stream = torch.cuda.Stream()
    for ends in ([0, 180, 300], [0, 100, 250], [7, 7, 40], [0, 0, 0], [0, 150, 300]):
        cu.copy_(torch.tensor(ends, dtype=torch.int32))
        for t in results:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        held = [torch.zeros_like(t) for t in results]
        pm.attention_forward(q, k, v, cu, out=held[0], lse=held[1])
        pm.attention_backward(do, q, k, v, held[0], held[1], cu, dq=held[2], dk=held[3], dv=held[4])
        torch.cuda.synchronize()
        apart = both(stream)
        torch.cuda.synchronize()
        for got, other, want in zip(results, apart, held):
            assert torch.equal(got, want) and torch.equal(other, want)


def test_heads_without_columns_are_refused():
    announce("attention heads of no columns")
    none = torch.empty((40, 1, 0), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    with pytest.raises(pm.MuonHError, match="dim"):
        pm.attention_forward(none, none, none, cu)


@pytest.mark.parametrize("heads,dim", SPLITS[:4])
def test_infinite_keys_by_the_sign_of_their_scores(heads, dim):
    """A key with an infinity: a later row whose score it makes -inf has what the formula
    gives without that key (NaN and lse -inf if it sees no other), one whose score it makes
    +inf is NaN, and earlier rows stay within the tolerances."""
    n = 150
    q, k, v, do, cu = _inputs([n], heads, heads, dim)
    assert (q != 0).all()
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    for where in (0, 5, 31, 32, 40, 64, 100, 149):
        for value in (float("inf"), -float("inf")):
            announce(f"attention key {value} at {where}, {heads} heads of {dim}")
            bad = k.clone()
            bad[where, :, 3] = value
            out, lse = pm.attention_forward(q, bad, v, cu)
            O, L, Q, K, V = (_np(t) for t in (out, lse, q, k, v))
            for h in {0, heads // 2, heads - 1}:
                seen = (j <= i) & (j != where)
                up = (np.arange(n) >= where) & (Q[:, h, 3] * value > 0)
                some = seen.any(axis=1) & ~up
                assert np.isnan(O[~some, h]).all() and np.isnan(L[h, up]).all() and (L[h, ~some & ~up] == -np.inf).all()
                want, wl, tol, ltol = _seen_softmax(Q[:, h], K[:, h], V[:, h], dim ** -0.5, seen)
                assert np.all(np.abs(O[some, h] - want[some]) <= tol[some]), (h, "out")
                assert np.all(np.abs(L[h, some] - wl[some]) <= ltol[some]), (h, "lse")


@pytest.mark.parametrize("heads,dim", SPLITS)
@pytest.mark.parametrize("scale", [0.5, 1.0])
def test_keys_masked_by_the_least_value(scale, heads, dim):
    """The first 70 keys have bf16's lowest value as their score, a finite number (with scale 1
    not so in units of log2 e): rows that see another key have what the formula gives without
    them."""
    announce(f"attention lowest scores, scale {scale}, {heads} heads of {dim}")
    n, masked = 200, 70
    q, k, v, do, cu = _inputs([n], heads, heads, dim, spread=0.2)
    q[:, :, -1] = 1.0
    k[:, :, -1] = 0.0
    clean = _np(k)
    k[:masked, :, -1] = torch.finfo(torch.bfloat16).min
    out, lse = pm.attention_forward(q, k, v, cu, scale=scale)
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    seen = (j <= i) & (j >= masked)
    O, L, Q, V = _np(out), _np(lse), _np(q), _np(v)
    for h in {0, heads // 2, heads - 1}:
        want, wl, tol, ltol = _seen_softmax(Q[:, h], clean[:, h], V[:, h], scale, seen)
        assert np.all(np.abs(O[masked:, h] - want[masked:]) <= tol[masked:]), (h, "out")
        assert np.all(np.abs(L[h, masked:] - wl[masked:]) <= ltol[masked:]), (h, "lse")


@pytest.mark.parametrize("heads,dim", SPLITS)
def test_rows_of_huge_scores(heads, dim):
    """Rows whose scores are all equal and far below zero, as those that a mask leaves
    nothing else, are the keys' mean; of scores that grow by 2^33 every 8 keys the last ones
    count; other rows of the same wavefronts have what the formula gives."""
    announce(f"attention huge scores, {heads} heads of {dim}")
    n = 200
    q, k, v, do, cu = _inputs([n], heads, heads, dim, spread=0.2)
    q[:, :, -1] = k[:, :, -1] = 0.0
    huge = torch.arange(n, device="cuda") % 3 == 1
    Q, plain, V = _np(q), _np(k), _np(v)
    for value in (torch.finfo(torch.bfloat16).min, -2.0 ** 30, 2.0 ** 30):
        bad = k.clone()
        bad[:, :, -1] = value
        if value > 0:
            bad[:, :, -1] *= 1 + torch.arange(n, device="cuda")[:, None] // 8 * 8   # whole in 8 bits
        mixed = q.clone()
        mixed[huge] = 0.0
        mixed[huge, :, -1] = 1.0
        out, lse = pm.attention_forward(mixed, bad, v, cu, scale=1.0)
        O, L, K = _np(out), _np(lse), _np(bad)[:, 0, -1]
        rest = ~_np(huge.float()).astype(bool)
        for h in {0, heads // 2, heads - 1}:
            want, wl, tol, ltol = _seen_softmax(Q[:, h], plain[:, h], V[:, h], 1.0, np.tril(np.ones((n, n), dtype=bool)))
            assert np.all(np.abs(O[rest, h] - want[rest]) <= tol[rest]), (value, h, "out")
            assert np.all(np.abs(L[h, rest] - wl[rest]) <= ltol[rest]), (value, h, "lse")
        for i in np.flatnonzero(_np(huge.float())):
            top = K[:i + 1] == K[:i + 1].max()
            mean, size = V[:i + 1][top].mean(axis=0), np.abs(V[:i + 1][top]).mean(axis=0)
            tol = size * 2 * n * U
            assert np.all(np.abs(O[i] - mean) <= tol + B * (np.abs(mean) + tol)), (value, i)
            assert np.all(np.abs(L[:, i] - (K[i] + np.log(top.sum()))) <= 2 * U * abs(K[i]) + 8 * U), (value, i)


@pytest.mark.parametrize("heads,dim", SPLITS)
@pytest.mark.parametrize("flag", [1.0, 8.0])
def test_gradients_of_rows_that_a_mask_leaves_nothing(flag, heads, dim):
    """Rows whose keys are all masked by the lowest number (scores finite, or -inf where q
    has 8) add nothing to the gradients and have none; the others have what the formula
    gives without the masked keys."""
    announce(f"attention gradients of masked rows, {flag}, {heads} heads of {dim}")
    n, masked = 300, 70
    q, k, v, do, cu = _inputs([n], heads, heads, dim, spread=0.2)
    q[:, :, -1] = flag
    k[:, :, -1] = 0.0
    clean = _np(k)
    k[:masked, :, -1] = torch.finfo(torch.bfloat16).min
    out, lse = pm.attention_forward(q, k, v, cu, scale=1.0)
    dq, dk, dv = (_np(t) for t in pm.attention_backward(do, q, k, v, out, lse, cu, scale=1.0))
    for t in (dq, dk, dv):
        assert (t[:masked] == 0).all()
    seen = np.tril(np.ones((n - masked, n - masked), dtype=bool))
    Q, V, DO, O, L = (_np(t)[masked:] if t.dim() == 3 else _np(t)[:, masked:] for t in (q, v, do, out, lse))
    K, m = clean[masked:], n - masked
    for h in {0, heads // 2, heads - 1}:
        a, b, vh, d = Q[:, h], K[:, h], V[:, h], DO[:, h]
        S = a @ b.T
        P = np.where(seen, np.exp(np.where(seen, S, 0.0) - L[h][:, None]), 0.0)
        ep = dim * U * (np.abs(a) @ np.abs(b).T) + 8 * U * (np.abs(S) + np.abs(L[h])[:, None] + 1)
        size = np.abs(d * O[:, h]).sum(axis=1, keepdims=True)
        delta = (d * O[:, h]).sum(axis=1, keepdims=True)
        dP = d @ vh.T
        ds = P * (dP - delta)
        eds = np.abs(ds) * (B + 2 * ep) + P * (dim * U * (np.abs(d) @ np.abs(vh).T + size) + 2 * U * np.abs(dP - delta))
        for name, got, want, tol in (
                ("dq", dq[masked:, h], ds @ b, eds @ np.abs(b) + 2 * m * U * (np.abs(ds) @ np.abs(b))),
                ("dk", dk[masked:, h], ds.T @ a, eds.T @ np.abs(a) + 2 * m * U * (np.abs(ds).T @ np.abs(a))),
                ("dv", dv[masked:, h], P.T @ d, (P * (B + 2 * ep + 2 * m * U)).T @ np.abs(d))):
            tol = tol + B * (np.abs(want) + tol)
            assert np.all(np.abs(got - want) <= tol), (name, h, float((np.abs(got - want) - tol).max()))


@pytest.mark.parametrize("heads,kv,dim", [(4, 2, 40), (4, 1, 104), (64, 32, 40), (120, 60, 104)])
def test_huge_scores_in_groups_of_heads(heads, kv, dim):
    """Two sequences and padding, heads that share keys, widths between the tiles': rows of
    equal scores far below zero are the mean of their own sequence's values up to them, also
    where a later value is NaN."""
    announce(f"attention huge scores, {heads}/{kv} heads of {dim}")
    lens, tail = [150, 71], 9
    q, k, v, do, cu = _inputs(lens, heads, kv, dim, tail=tail)
    q[:], k[:] = 0.0, 0.0
    q[:, :, 0], k[:, :, 0] = 1.0, -2.0 ** 100
    v[140] = float("nan")
    out, lse = pm.attention_forward(q, k, v, cu, scale=1.0)
    O, L, V = _np(out), _np(lse), _np(v)
    assert np.isnan(O[140:150]).all() and (L[:, :221] == -2.0 ** 100).all() and (L[:, 221:] == 0).all()
    for start, rows in ((0, 140), (150, 71)):
        part = np.repeat(V[start:start + rows], heads // kv, axis=1)
        n = np.arange(1, rows + 1)[:, None, None]
        mean, size = part.cumsum(axis=0) / n, np.abs(part).cumsum(axis=0) / n
        tol = 2 * n * U * size
        assert np.all(np.abs(O[start:start + rows] - mean) <= tol + B * (np.abs(mean) + tol))


def test_zeros_into_slices_from_c():
    """The C entry points' zero_rest: each bit clears its own result's rows, within the
    heads' columns of a fused buffer."""
    announce("attention zero_rest into slices")
    lib, byref = pm.load_library(), ctypes.byref
    heads, kv, dim, lens, tail = 4, 2, 72, [33, 140], 50
    q, k, v, do, cu = _inputs(lens, heads, kv, dim, tail=tail)
    n, live = len(q), sum(lens)
    want, wl = pm.attention_forward(q, k, v, cu)
    wants = (want, wl.T) + pm.attention_backward(do, q, k, v, want, wl, cu)
    stream = torch.cuda.current_stream().cuda_stream
    for bits in range(32):
        wide = torch.full((n, (2 * heads + 2 * kv) * dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        parts = [t.unflatten(1, (-1, dim)) for t in wide[:, :-8].split([heads * dim, heads * dim, kv * dim, kv * dim], 1)]
        lse = torch.full((heads, n), 7.0, device="cuda")
        ld = wide.stride(0)
        args = mb.muonh_attention_args(q.data_ptr(), k.data_ptr(), v.data_ptr(), parts[0].data_ptr(), lse.data_ptr(), cu.data_ptr(), n,
                                       2, heads * dim, kv * dim, kv * dim, ld, heads, kv, dim, dim ** -0.5, bits)
        assert lib.muonh_attention_forward(byref(args), stream) == 0
        ws = torch.empty(2 * heads * n + 128, device="cuda")
        grad = mb.muonh_attention_grad_args(args, do.data_ptr(), *(t.data_ptr() for t in parts[1:]), heads * dim, ld, ld, ld,
                                            ws.data_ptr(), ws.numel() * 4)
        assert lib.muonh_attention_backward(byref(grad), stream) == 0
        for i, (got, clean) in enumerate(zip((parts[0], lse.T, *parts[1:]), wants)):
            assert torch.equal(got[:live], clean[:live])
            assert (got[live:] == (0 if bits >> i & 1 else 7)).all(), (bits, i)
        assert (wide[:, -8:] == 7).all()
