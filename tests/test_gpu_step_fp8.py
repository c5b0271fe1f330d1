"""muonh_step_quantized against muonh_step followed by fp8_quantize, bit for bit,
and a training step of one layer through every operator (MI355X only)."""

import numpy as np
import pytest
import torch

import oracle
import pretraining_optimizer_amd as pm
from oracle import block_fp8, norm
from parity import announce

pytestmark = pytest.mark.gpu

SHAPES = [(300, 200), (128, 640), (515, 129), (1, 77), (256, 256), (130, 1030)]


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _setup(shapes, gdt, seed):
    gen = torch.Generator().manual_seed(seed)
    ws = [torch.randn(s, generator=gen).cuda() for s in shapes]
    gs = [[torch.randn(s, generator=gen).to(gdt).cuda() for s in shapes] for _ in range(3)]
    return ws, gs


def _same(a, b):
    return torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scale, b.scale)


@pytest.mark.parametrize("ns,gdt,mode", [("bf16", torch.bfloat16, pm.MUONH_MODE_HYPERBALL),
                                         ("f32", torch.float32, pm.MUONH_MODE_HYPERBALL),
                                         ("bf16", torch.float32, pm.MUONH_MODE_MUON_WD)])
def test_step_writes_the_updated_weights_forms(ns, gdt, mode):
    announce(f"quantised step {ns} {gdt} mode {mode}")
    ws, gs = _setup(SHAPES, gdt, 7)
    opts = dict(grad_dtype=gdt, ns_dtype=pm.MUONH_BF16 if ns == "bf16" else pm.MUONH_F32, mode=mode, weight_decay=0.1)
    ref = [w.clone() for w in ws]
    ms, mr = [torch.zeros_like(w) for w in ws], [torch.zeros_like(w) for w in ws]
    a, b = pm.MuonH(ws, ms, **opts), pm.MuonH(ref, mr, **opts)
    fp8 = [pm.fp8_quantize(w, form="both", block_rows=128) for w in ws]
    fp8[1] = (fp8[1][0], None)
    fp8[4] = None
    before = [None if p is None else p[0].data.view(torch.uint8).clone() for p in fp8]
    for k in range(3):
        if k == 2:   # other outputs than before
            fp8[0] = (pm.Fp8Matrix.empty(*SHAPES[0], 128), pm.Fp8Matrix.empty(*SHAPES[0][::-1], 128))
        a.step(gs[k], elr=0.02, fp8=fp8)
        b.step(gs[k], elr=0.02)
        for i, pair in enumerate(fp8):
            assert torch.equal(ws[i], ref[i]) and torch.equal(ms[i], mr[i]), (k, i)
            q, qt = pm.fp8_quantize(ref[i], form="both", block_rows=128)
            if pair is None:
                continue
            assert _same(pair[0], q), (k, i)
            assert pair[1] is None or _same(pair[1], qt), (k, i)
    assert any(not torch.equal(x, p[0].data.view(torch.uint8)) for x, p in zip(before, fp8) if p is not None)
    assert a.stats() == b.stats()
    # a plain step in between, on another stream
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.step(gs[0], elr=0.01, stream=s)
    a.step(gs[1], elr=0.01, stream=s, fp8=fp8)
    torch.cuda.current_stream().wait_stream(s)
    b.step(gs[0], elr=0.01)
    b.step(gs[1], elr=0.01)
    assert torch.equal(ws[2], ref[2]) and _same(fp8[2][1], pm.fp8_quantize(ref[2], form="col", block_rows=128))
    a.close()
    b.close()


def test_step_with_non_finite_gradient():
    """A NaN gradient makes a NaN weight, whose forms are NaN everywhere."""
    w, m = torch.randn((200, 130), device="cuda"), torch.zeros((200, 130), device="cuda")
    opt = pm.MuonH([w], [m], grad_dtype=torch.float32)
    g = torch.randn((200, 130), device="cuda")
    g[3, 3] = float("nan")
    q, qt = pm.fp8_quantize(w, form="both", block_rows=128)
    opt.step([g], elr=0.01, fp8=[(q, qt)])
    assert opt.stats()[0]["nonfinite"] == 1 and torch.isnan(w).all()
    assert torch.isnan(q.data.float()[:, :130]).all() and torch.isnan(qt.data.float()[:, :200]).all()
    assert not q.data.float()[:, 130:].any() and not qt.data.float()[:, 200:].any()
    opt.close()


def test_step_refusals():
    w, m = torch.randn((200, 130), device="cuda"), torch.zeros((200, 130), device="cuda")
    g = torch.randn((200, 130), device="cuda")
    opt = pm.MuonH([w], [m], grad_dtype=torch.float32)
    keep = w.clone()
    good = pm.fp8_quantize(w, form="both", block_rows=128)
    with pytest.raises(ValueError):
        opt.step([g], elr=0.01, fp8=[good, good])
    with pytest.raises(ValueError):
        opt.step([g], elr=0.01, fp8=[good], graph=True)
    for bad in ((good[1], None), (None, good[0]), (pm.fp8_quantize(w), None)):
        with pytest.raises(pm.MuonHError):
            opt.step([g], elr=0.01, fp8=[bad])
    w2, m3 = torch.randn((200, 130), device="cuda"), torch.zeros((200, 130), device="cuda")
    two = pm.MuonH([w, w2], [m, m3], grad_dtype=torch.float32)
    with pytest.raises(pm.MuonHError, match="twice"):
        two.step([g, g], elr=0.01, fp8=[good, good])
    two.close()
    assert torch.equal(w, keep)
    opt.step([g], elr=0.01, fp8=[(None, None)])   # nothing to write: the plain update
    other = keep.clone()
    m2 = torch.zeros_like(m)
    ref = pm.MuonH([other], [m2], grad_dtype=torch.float32)
    ref.step([g], elr=0.01)
    assert torch.equal(w, other)
    opt.close()
    ref.close()


def test_step_is_refused_while_the_stream_is_captured():
    w, m = torch.randn((200, 130), device="cuda"), torch.zeros((200, 130), device="cuda")
    g = torch.randn((200, 130), device="cuda")
    opt = pm.MuonH([w], [m], grad_dtype=torch.float32)
    forms = pm.fp8_quantize(w, form="both", block_rows=128)
    keep, x = w.clone(), torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1.0)
        with pytest.raises(pm.MuonHError, match="captured"):
            opt.step([g], elr=0.01, fp8=[forms])
    graph.replay()
    assert torch.equal(w, keep) and x.sum().item() == 4.0
    opt.step([g], elr=0.01, fp8=[forms])   # outside it is an ordinary step
    q, qt = pm.fp8_quantize(w, form="both", block_rows=128)
    assert not torch.equal(w, keep) and _same(forms[0], q) and _same(forms[1], qt)
    opt.close()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_layer_training_steps(kind):
    """h = norm(x) W^T trained for three steps on sum (h - target)^2 / 2: norm,
    products in FP8, gradients, MuonH with FP8 weights, AdamW for the norm.

    Each stage is checked from the tensors the previous one left: the products'
    gradients against the unquantised formula (both factors of a product are
    within 2^-4 of their values, or within 2^-10 of their block's scale, so a
    term is off by at most 2 2^-4 + 2^-8 of itself and the scales' share), the
    forward product against the oracle's on the same FP8 operands."""
    announce(f"layer steps {kind}")
    tokens, d, out = 300, 260, 390
    gen = torch.Generator().manual_seed(3)
    x = (torch.randn((tokens, d), generator=gen) * 2 + 0.3).bfloat16().cuda()
    target = torch.randn((tokens, out), generator=gen).cuda()
    w = (torch.randn((out, d), generator=gen) / d ** 0.5).cuda()
    gamma = torch.ones(d, device="cuda")
    beta = torch.zeros(d, device="cuda") if kind == "layer" else None
    mw = torch.zeros_like(w)
    muon = pm.MuonH([w], [mw], grad_dtype=torch.float32, ns_dtype=pm.MUONH_F32)
    vecs = [gamma] + ([beta] if beta is not None else [])
    adam = pm.AdamW(vecs, [torch.zeros_like(v) for v in vecs], [torch.zeros_like(v) for v in vecs], grad_dtype=torch.float32)
    wq, wqt = pm.fp8_quantize(w, form="both", block_rows=128)
    state = oracle.OracleMatrixState.from_arrays(_np(w))
    for k in range(3):
        y, mean, rstd = pm.norm_forward(x, gamma, beta, kind=kind)
        yr, yc = pm.fp8_quantize(y, form="both")
        h = pm.fp8_matmul(yr, wq, out_dtype=torch.float32)
        dh = (h - target).bfloat16()
        hr, hc = pm.fp8_quantize(dh, form="both")
        dy = pm.fp8_matmul(hr, wqt)
        dw = pm.fp8_matmul(hc, yc, out_dtype=torch.float32)
        dx, dgamma, dbeta = pm.norm_backward(dy, x, gamma, mean, rstd, kind=kind, bias=beta is not None)

        Y, W, D = _np(y), _np(w), _np(dh)
        want = block_fp8.matmul(block_fp8.quantize(Y), block_fp8.quantize(W, 128))
        scale = np.abs(Y) @ np.abs(W).T * 2.0
        assert np.all(np.abs(_np(h) - want) <= d * 2.0 ** -23 * scale)

        def near(got, p, q, step):
            # p's and q's smallest steps: 2^-10 of a block's scale, at most 2^-10 (amax / 224)
            term = np.abs(p) @ np.abs(q)
            share = (np.abs(p).max() / 224 * 2.0 ** -10) * np.abs(q).sum(0)[None, :] + \
                    (np.abs(q).max() / 224 * 2.0 ** -10) * np.abs(p).sum(1)[:, None]
            assert np.all(np.abs(got - p @ q) <= (2 * 2.0 ** -4 + 2.0 ** -8 + step) * term + 1.1 * share)

        near(_np(dy), D, W, 2.0 ** -8 + 7 * 2.0 ** -13 + out * 2.0 ** -23)
        near(_np(dw), D.T, Y, tokens * 2.0 ** -23)
        rdx, rdg, rdb = norm.norm_backward(_np(dy), _np(x), _np(gamma), _np(mean), _np(rstd), kind)
        assert np.linalg.norm(_np(dx) - rdx) <= 2.0 ** -8 * np.linalg.norm(rdx)
        assert np.allclose(_np(dgamma), rdg, rtol=1e-5, atol=1e-5 * np.abs(rdg).max())
        if beta is not None:
            assert np.allclose(_np(dbeta), rdb, rtol=1e-5, atol=1e-5 * np.abs(rdb).max())

        muon.step([dw], elr=0.02, fp8=[(wq, wqt)])
        adam.step([dgamma] + ([dbeta] if beta is not None else []), 1e-2, k + 1)
        oracle.muonh_step([state], [_np(dw)], 0.02)
        # the parity gate of one fp32 step, for each step so far
        assert np.linalg.norm(_np(w) - state.w) <= (k + 1) * (2 * 0.02 * 1e-4 + 1e-5) * np.linalg.norm(state.w)
        q, qt = pm.fp8_quantize(w, form="both", block_rows=128)
        assert _same(wq, q) and _same(wqt, qt)
    muon.close()
    adam.close()
