"""The step that writes FP8 weights on each plan, mode and option of the step it
extends: bit for bit the plain step followed by fp8_quantize (MI355X only)."""

import pytest
import torch

import pretraining_optimizer_amd as pm
from parity import announce

pytestmark = pytest.mark.gpu

LARGE = [(2048, 6144), (6144, 2048), (2001, 1999), (300, 5000), (4100, 129)]
SMALL = [(256, 128), (77, 1), (1, 300), (129, 257)]
MODES = [pm.MUONH_MODE_HYPERBALL, pm.MUONH_MODE_MUON_WD, pm.MUONH_MODE_ELR_ALIGNED]


def _same(a, b):
    return torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scale, b.scale)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shapes,ns,tile", [(LARGE, pm.MUONH_BF16, None), (LARGE, pm.MUONH_F32, None), (SMALL, pm.MUONH_BF16, "256"),
                                            (SMALL, pm.MUONH_F32, "64"), (LARGE[2:], pm.MUONH_BF16, "64")])
def test_every_plan_and_mode(shapes, ns, tile, mode, monkeypatch):
    announce(f"quantised step {len(shapes)} matrices ns {ns} tile {tile} mode {mode}")
    if tile is not None:
        monkeypatch.setenv("MUONH_GEMM_TILE", tile)
    gen = torch.Generator(device="cuda").manual_seed(5)
    ws = [torch.randn(s, generator=gen, device="cuda") for s in shapes]
    ref = [w.clone() for w in ws]
    ms, mr = [torch.zeros_like(w) for w in ws], [torch.zeros_like(w) for w in ws]
    opts = dict(grad_dtype=torch.bfloat16, ns_dtype=ns, mode=mode, weight_decay=0.1, nesterov=1)
    a, b = pm.MuonH(ws, ms, **opts), pm.MuonH(ref, mr, **opts)
    fp8 = [(pm.Fp8Matrix.empty(*s, 128), pm.Fp8Matrix.empty(s[1], s[0], 128)) for s in shapes]
    scale = [0.5 + 0.25 * i for i in range(len(shapes))]
    for k in range(2):
        gs = [torch.randn(s, generator=gen, device="cuda").bfloat16() for s in shapes]
        a.step(gs, elr=0.02, elr_scale=scale, fp8=fp8)
        b.step(gs, elr=0.02, elr_scale=scale)
        for i, (q, qt) in enumerate(fp8):
            assert torch.equal(ws[i], ref[i]) and torch.equal(ms[i], mr[i]), (k, i)
            want, want_t = pm.fp8_quantize(ref[i], form="both", block_rows=128)
            assert _same(q, want) and _same(qt, want_t), (k, i)
    assert a.stats() == b.stats()
    # a recorded plain step in between leaves the forms as they were
    keep = [q.data.view(torch.uint8).clone() for q, _ in fp8]
    a.step(gs, elr=0.01, graph=True)
    b.step(gs, elr=0.01, graph=True)
    assert all(torch.equal(q.data.view(torch.uint8), k) for (q, _), k in zip(fp8, keep))
    a.step(gs, elr=0.01, fp8=fp8)
    b.step(gs, elr=0.01)
    for i, (q, qt) in enumerate(fp8):
        want, want_t = pm.fp8_quantize(ref[i], form="both", block_rows=128)
        assert torch.equal(ws[i], ref[i]) and _same(q, want) and _same(qt, want_t), i
    a.close()
    b.close()


def test_outputs_change_between_streams():
    """Steps on two streams in turn whose outputs change each time: each waits for
    the one before, and its table is uploaded only then."""
    announce("quantised step on two streams")
    shapes = [(1024, 1024), (700, 1500)]
    ws = [torch.randn(s, device="cuda") for s in shapes]
    ref = [w.clone() for w in ws]
    gs = [torch.randn(s, device="cuda").bfloat16() for s in shapes]
    a = pm.MuonH(ws, [torch.zeros_like(w) for w in ws])
    b = pm.MuonH(ref, [torch.zeros_like(w) for w in ref])
    sets = [[(pm.Fp8Matrix.empty(*s, 128), pm.Fp8Matrix.empty(s[1], s[0], 128)) for s in shapes] for _ in range(6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for k, fp8 in enumerate(sets):
        a.step(gs, elr=0.01, stream=streams[k % 2], fp8=fp8)
    torch.cuda.synchronize()
    for k, fp8 in enumerate(sets):
        b.step(gs, elr=0.01)
        for i, (q, qt) in enumerate(fp8):
            want, want_t = pm.fp8_quantize(ref[i], form="both", block_rows=128)
            assert _same(q, want) and _same(qt, want_t), (k, i)
    assert all(torch.equal(w, r) for w, r in zip(ws, ref))
    a.close()
    b.close()
