"""Attention, residual norm, embedding, FP8 products and the optimizers together, as
the layers of a model use them (MI355X only): training steps whose every stage is
checked against the fp64 oracles, and their forward and backward passes as a graph."""

import numpy as np
import pytest
import torch

import pretraining_optimizer_amd as pm
import test_gpu_add_norm as residual_norm
import test_gpu_attention as attention
import test_gpu_embedding as embedding
from oracle import block_fp8, norm
from parity import announce

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -23, 2.0 ** -8
ROWS, DIM, HEADS, KV, WIDTH, OUT, LAYERS = 500, 40, 6, 2, 264, 390, 2
LENS = [100, 1, 0, 133, 66]
TOKENS = sum(LENS)
SCALE = WIDTH ** 0.5


def _np(t):
    return t.detach().double().cpu().numpy()


class Model:
    """h_0 = embedding; h_{l+1} = h_l + W_o attention(W_qkv norm(h_l)); the loss is
    sum (W_out norm(h_L) - target)^2 / 2."""

    def __init__(self, seed=3):
        gen = torch.Generator().manual_seed(seed)

        def make(*shape, std):
            return (std * torch.randn(shape, generator=gen)).cuda()

        self.table = make(ROWS, WIDTH, std=WIDTH ** -0.5)
        self.gammas = [1.0 + make(WIDTH, std=0.1) for _ in range(LAYERS + 1)]
        self.weights = [w for _ in range(LAYERS) for w in (make((HEADS + 2 * KV) * DIM, WIDTH, std=WIDTH ** -0.5),
                                                          make(WIDTH, HEADS * DIM, std=(HEADS * DIM) ** -0.5))]
        self.weights.append(make(OUT, WIDTH, std=WIDTH ** -0.5))
        self.forms = [pm.fp8_quantize(w, form="both", block_rows=128) for w in self.weights]
        self.target = make(TOKENS, OUT, std=1.0)
        self.tokens = torch.randint(0, ROWS // 2, (TOKENS,), generator=gen)
        self.tokens[::9] = -1   # padding
        self.tokens = self.tokens.cuda()
        self.cu = torch.tensor([0] + list(np.cumsum(LENS)), dtype=torch.int32, device="cuda")

    def split(self, t):
        return t.unflatten(1, (HEADS + 2 * KV, DIM)).split((HEADS, KV, KV), 1)

    def forward(self):
        s = {"layers": []}
        h = s["x"] = pm.embedding_forward(self.tokens, self.table, scale=SCALE)
        a = None
        for i in range(LAYERS):
            layer = {"a": a, "before": h}
            h, layer["rstd"], layer["n"] = (pm.add_norm_quantize(h, None, self.gammas[i], form="both") if a is None else
                                            pm.add_norm_quantize(a, h, self.gammas[i], form="both"))
            layer["h"] = h
            layer["qkv"] = pm.fp8_matmul(layer["n"][0], self.forms[2 * i][0])
            layer["out"], layer["lse"] = pm.attention_forward(*self.split(layer["qkv"]), self.cu)
            layer["o"] = pm.fp8_quantize(layer["out"].flatten(1), form="both")
            a = pm.fp8_matmul(layer["o"][0], self.forms[2 * i + 1][0])
            s["layers"].append(layer)
        s["a"], s["before"] = a, h
        s["h"], s["rstd"], s["n"] = pm.add_norm_quantize(a, h, self.gammas[-1], form="both")
        s["y"] = pm.fp8_matmul(s["n"][0], self.forms[-1][0], out_dtype=torch.float32)
        return s

    def backward(self, s):
        g = {"layers": [None] * LAYERS, "weights": [None] * len(self.weights), "gammas": [None] * (LAYERS + 1)}
        g["dy"] = (s["y"] - self.target).bfloat16()
        dyr, dyc = pm.fp8_quantize(g["dy"], form="both")
        g["dn"] = pm.fp8_matmul(dyr, self.forms[-1][1])
        g["weights"][-1] = pm.fp8_matmul(dyc, s["n"][1], out_dtype=torch.float32)
        dh, g["gammas"][-1], _ = pm.norm_backward(g["dn"], s["h"], self.gammas[-1], None, s["rstd"])
        g["dh"] = dh
        for i in reversed(range(LAYERS)):
            layer, d = s["layers"][i], {"above": dh}
            dar, dac = pm.fp8_quantize(dh, form="both")
            g["weights"][2 * i + 1] = pm.fp8_matmul(dac, layer["o"][1], out_dtype=torch.float32)
            d["dout"] = pm.fp8_matmul(dar, self.forms[2 * i + 1][1]).unflatten(1, (HEADS, DIM))
            d["dqkv"] = torch.empty_like(layer["qkv"])
            dq, dk, dv = self.split(d["dqkv"])
            pm.attention_backward(d["dout"], *self.split(layer["qkv"]), layer["out"], layer["lse"], self.cu, dq=dq, dk=dk, dv=dv)
            dr, dc = pm.fp8_quantize(d["dqkv"], form="both")
            g["weights"][2 * i] = pm.fp8_matmul(dc, layer["n"][1], out_dtype=torch.float32)
            d["dn"] = pm.fp8_matmul(dr, self.forms[2 * i][1])
            dh, g["gammas"][i] = pm.add_norm_backward(d["dn"], dh, layer["h"], self.gammas[i], layer["rstd"])
            d["dh"] = dh
            g["layers"][i] = d
        g["table"] = pm.embedding_backward(self.tokens, dh, ROWS, scale=SCALE)
        return g


def _check_product(got, a, w, width, what):
    """A product of FP8 operands a and quantised w, whose sums are of `width` terms."""
    want = block_fp8.matmul(a, block_fp8.quantize(w, 128))
    size = np.abs(a.dequantize()) @ np.abs(block_fp8.quantize(w, 128).dequantize()).T
    tol = width * U * size
    if got.dtype == torch.bfloat16:
        tol = tol + B * (np.abs(want) + tol)
    assert np.all(np.abs(_np(got) - want) <= tol), what


def _check_near(got, p, q, width, what):
    """p q of operands that were quantised in blocks: each factor of a product is within
    2^-4 of its value, or within 2^-10 of its block's scale (at most amax / 224)."""
    term = np.abs(p) @ np.abs(q)
    share = np.abs(p).max() / 224 * 2.0 ** -10 * np.abs(q).sum(0)[None, :] + \
        np.abs(q).max() / 224 * 2.0 ** -10 * np.abs(p).sum(1)[:, None]
    step = 2 * 2.0 ** -4 + 2.0 ** -8 + width * U + (2.0 ** -8 + 2.0 ** -11 if got.dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(_np(got) - p @ q) <= step * term + 1.1 * share), what


def _check_step(m, s, g):
    x = _np(s["x"])
    known = _np(m.tokens) >= 0
    rows = _np(m.table)[m.tokens.clamp(min=0).cpu().numpy()] * known[:, None]
    assert np.all(np.abs(x - SCALE * rows) <= (B + 4 * U) * np.abs(SCALE * rows)) and not x[~known].any()
    for i in range(LAYERS + 1):
        layer = s["layers"][i] if i < LAYERS else s
        a, before, gamma = layer["a"], layer["before"], m.gammas[i]
        residual_norm._check_forward(before if a is None else a, None if a is None else before, gamma, 1e-6,
                                     (layer["h"], layer["rstd"], layer["n"]), "both", f"norm {i}")
        y = _np((layer["h"].float() * layer["rstd"][:, None]) * gamma)
        w = _np(m.weights[2 * i])
        _check_product(layer["qkv"] if i < LAYERS else layer["y"], block_fp8.quantize(y), w, WIDTH, f"product {i}")
        d = g["layers"][i] if i < LAYERS else g
        dy = _np(d["dqkv"] if i < LAYERS else d["dy"])
        _check_near(d["dn"], dy, w, w.shape[0], f"dn {i}")
        _check_near(g["weights"][2 * i], dy.T, y, TOKENS, f"dw {2 * i}")
        if i == LAYERS:
            rdx, rdg, _ = norm.norm_backward(_np(d["dn"]), _np(s["h"]), _np(gamma), None, _np(s["rstd"]), "rms")
            assert np.linalg.norm(_np(d["dh"]) - rdx) <= B * np.linalg.norm(rdx)
            assert np.allclose(_np(g["gammas"][i]), rdg, rtol=1e-5, atol=1e-5 * np.abs(rdg).max())
            continue
        residual_norm._check_backward((d["dh"], g["gammas"][i]), d["dn"], d["above"], layer["h"], gamma, layer["rstd"],
                                      torch.bfloat16, f"norm back {i}")
        q, k, v = m.split(layer["qkv"])
        attention._check_forward(layer["out"], layer["lse"], q, k, v, m.cu, DIM ** -0.5, f"attention {i}")
        attention._check_backward(m.split(d["dqkv"]), d["dout"], q, k, v, layer["out"], layer["lse"], m.cu, DIM ** -0.5,
                                  f"attention back {i}")
        o, w = _np(layer["out"].flatten(1)), _np(m.weights[2 * i + 1])
        a = s["layers"][i + 1]["a"] if i + 1 < LAYERS else s["a"]
        _check_product(a, block_fp8.quantize(o), w, HEADS * DIM, f"output product {i}")
        _check_near(d["dout"].flatten(1), _np(d["above"]), w, WIDTH, f"dout {i}")
        _check_near(g["weights"][2 * i + 1], _np(d["above"]).T, o, TOKENS, f"dw {2 * i + 1}")
    embedding._check_backward(g["table"], m.tokens, g["layers"][0]["dh"], ROWS, SCALE, "embedding back")


def _results(s, g):
    """Every tensor of a step, in one order."""
    out = []

    def walk(t):
        if isinstance(t, torch.Tensor):
            out.append(t)
        elif isinstance(t, pm.Fp8Matrix):
            out.extend([t.data.view(torch.uint8), t.scale])
        elif isinstance(t, dict):
            for key in sorted(t):
                walk(t[key])
        elif t is not None:
            for x in t:
                walk(x)

    walk(s)
    walk(g)
    return out


def _optimizers(m):
    muon = pm.MuonH(m.weights, [torch.zeros_like(w) for w in m.weights], grad_dtype=torch.float32)
    vectors = m.gammas + [m.table]
    adam = pm.AdamW(vectors, [torch.zeros_like(v) for v in vectors], [torch.zeros_like(v) for v in vectors],
                    grad_dtype=torch.float32)
    return muon, adam


def test_training_steps():
    announce("training steps of two layers")
    m = Model()
    muon, adam = _optimizers(m)
    unseen = torch.ones(ROWS, dtype=torch.bool, device="cuda")
    unseen[m.tokens.clamp(min=0)] = False
    unseen[0] = not bool((m.tokens == 0).any())
    decay = adam.options.weight_decay
    for k in range(2):
        s = m.forward()
        g = m.backward(s)
        _check_step(m, s, g)
        keep, radii = m.table.clone(), [w.norm() for w in m.weights]
        muon.step(g["weights"], elr=0.02, fp8=m.forms)
        adam.step(g["gammas"] + [g["table"]], 1e-2, k + 1)
        # rows that no token names have no gradient, only the decay
        assert unseen.any() and not g["table"][unseen].any()
        assert torch.allclose(m.table[unseen], keep[unseen] * (1 - 1e-2 * decay), rtol=2.0 ** -22, atol=0)
        assert not torch.equal(m.table[~unseen], keep[~unseen])
        for w, r, (q, qt) in zip(m.weights, radii, m.forms):
            assert torch.allclose(w.norm(), r, rtol=1e-5)
            a, b = pm.fp8_quantize(w, form="both", block_rows=128)
            for x, y in ((a, q), (b, qt)):
                assert torch.equal(x.data.view(torch.uint8), y.data.view(torch.uint8)) and torch.equal(x.scale, y.scale)
    muon.close()
    adam.close()


def test_passes_as_a_graph_between_steps():
    """The captured passes read the weights that eager steps update, and each replay
    equals the eager passes of a second model."""
    announce("captured passes of two layers")
    m, ref = Model(), Model()
    opts, ref_opts = _optimizers(m), _optimizers(ref)
    m.backward(m.forward())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = m.forward()
        g = m.backward(s)
    for k in range(4):
        graph.replay()
        rs = ref.forward()
        rg = ref.backward(rs)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(_results(s, g), _results(rs, rg))):
            assert torch.equal(x, y), (k, i, x.shape)
        for model, grads, (muon, adam) in ((m, g, opts), (ref, rg, ref_opts)):
            muon.step(grads["weights"], elr=0.02, fp8=model.forms)
            adam.step(grads["gammas"] + [grads["table"]], 1e-2, k + 1)
        # the target and the tokens change in place
        for model in (m, ref):
            model.target.mul_(0.5)
            model.tokens.copy_(model.tokens.roll(1))
    for pair in (opts, ref_opts):
        for o in pair:
            o.close()
