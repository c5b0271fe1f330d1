"""Cases, plain forms and 64-bit definitions of the FP8 and norm operators.

Four operators, as a training step of the matrices that the optimizer wraps
uses them:

  quantize   x -> E4M3 values and one power-of-two scale per block, as rows
             (the contraction runs along x's columns), as columns (along its
             rows: x transposed) or both; blocks of 1 x 128 for activations
             and gradients, of 128 x 128 for weights
  matmul     C = A B^T of two such operands, in bf16 or fp32
  norm       layer norm or RMS norm over the last axis, with its statistics
  norm_back  its gradients: dx, and dweight / dbias summed over the rows

With ``own`` False ``run`` computes them with elementary torch operations,
with ``own`` True through pretraining_optimizer_amd.  The layout of an FP8
operand: values [rows, ld] with ld = cols rounded up to 128 and zeros behind
the columns; scale exponents [rows or ceil(rows / 128), ld / 128 rounded up
to 4] as bytes, value = q * 2^(byte - 127), zero bytes behind the last block.
"""

import math

import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # activations of 2 sequences of 4096 tokens, for the forward and the weight-gradient product
        {"name": "quantize activations 8192x2048", "op": "quantize", "rows": 8192, "cols": 2048, "dtype": "bf16", "block": 1, "form": "both"},
        # an fp32 gradient with odd sizes, last groups cut on both axes
        {"name": "quantize gradient 1000x777", "op": "quantize", "rows": 1000, "cols": 777, "dtype": "f32", "block": 1, "form": "both"},
        # an fp32 master weight of the 1.7B set, once a step
        {"name": "quantize weight 6144x2048", "op": "quantize", "rows": 6144, "cols": 2048, "dtype": "f32", "block": 128, "form": "both"},
        # the forward product of the fused gate and up projections, the largest of the layer
        {"name": "matmul forward 8192x12288x2048", "op": "matmul", "m": 8192, "n": 12288, "k": 2048, "block": 128, "out": "bf16"},
        # a weight gradient, contracted over the tokens
        {"name": "matmul weight gradient 2048x6144x8192", "op": "matmul", "m": 2048, "n": 6144, "k": 8192, "block": 1, "out": "f32"},
        # the smallest call: one token through a down projection
        {"name": "matmul one token 1x2048x6144", "op": "matmul", "m": 1, "n": 2048, "k": 6144, "block": 128, "out": "bf16"},
        # odd sizes on every axis
        {"name": "matmul ragged 1000x777x1500", "op": "matmul", "m": 1000, "n": 777, "k": 1500, "block": 1, "out": "f32"},
        # the norm before a projection of the 1.7B set
        {"name": "norm rms 8192x2048", "op": "norm", "rows": 8192, "cols": 2048, "dtype": "bf16", "kind": "rms", "bias": False},
        # a few rows of odd length, where latency counts
        {"name": "norm layer 37x777", "op": "norm", "rows": 37, "cols": 777, "dtype": "f32", "kind": "layer", "bias": True},
        # its gradients in training
        {"name": "norm_back rms 8192x2048", "op": "norm_back", "rows": 8192, "cols": 2048, "dtype": "bf16", "kind": "rms", "bias": False},
        # norms of single heads: short rows, many of them
        {"name": "norm_back heads 131072x128", "op": "norm_back", "rows": 131072, "cols": 128, "dtype": "bf16", "kind": "rms", "bias": False},
        # long odd rows, few of them, with a bias
        {"name": "norm_back layer 300x5001", "op": "norm_back", "rows": 300, "cols": 5001, "dtype": "f32", "kind": "layer", "bias": True},
    ]


def _log(rng, low, high):
    """A whole number spread over the logarithm of its range, odd ones and multiples of 128 among them."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v > 256 and rng.random() < 0.5:
        v = (v + 64) // 128 * 128
    return min(max(v, low), high)


def draw(rng):
    op = rng.choice(["quantize", "matmul", "norm", "norm_back"])
    if op == "matmul":
        while True:
            m, n, k = _log(rng, 1, 16384), _log(rng, 1, 16384), _log(rng, 1, 16384)
            if m * n * k <= 8192 * 12288 * 2048:
                break
        return {"op": op, "m": m, "n": n, "k": k, "block": rng.choice([1, 128]), "out": rng.choice(["bf16", "f32"])}
    # a norm of a few values has a gradient of nothing but rounding: rows of 32 values and more
    least = 1 if op == "quantize" else 32
    while True:
        rows, cols = _log(rng, 1, 131072), _log(rng, least, 16384)
        if rows * cols <= 8192 * 2048:
            break
    case = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"])}
    if op == "quantize":
        return {**case, "block": rng.choice([1, 128]), "form": rng.choice(["row", "col", "both"])}
    return {**case, "kind": rng.choice(["layer", "rms"]), "bias": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs


def _values(gen, rows, cols, spread):
    """Normal values whose columns have scales of their own, as activations and gradients have."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    return x * torch.exp(spread * torch.randn((1, cols), generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        scale = 0.02 if case["block"] == 128 else 1.0
        x = scale * _values(gen, case["rows"], case["cols"], 0.0 if case["block"] == 128 else 1.0)
        return {**case, "x": x.to(TYPES[case["dtype"]])}
    if op == "matmul":
        a = _quantize(_values(gen, case["m"], case["k"], 0.5), 1)
        b = _quantize(0.02 * _values(gen, case["n"], case["k"], 0.0), case["block"])
        return {**case, "a": a[0], "sa": a[1], "b": b[0], "sb": b[1]}
    rows, cols, dtype = case["rows"], case["cols"], TYPES[case["dtype"]]
    state = {**case, "x": (_values(gen, rows, cols, 0.5) + 0.1).to(dtype),
             "weight": 1.0 + 0.1 * torch.randn(cols, generator=gen, device="cuda"),
             "b": 0.1 * torch.randn(cols, generator=gen, device="cuda") if case["bias"] else None}
    if op == "norm_back":
        # what the forward pass left: its statistics
        mean, rstd = _statistics(state["x"].double(), case["kind"])
        state["mean"], state["rstd"] = None if mean is None else mean.float().view(-1), rstd.float().view(-1)
        state["dy"] = (1e-2 * torch.randn((rows, cols), generator=gen, device="cuda")).to(dtype)
    return state


# ---------------------------------------------------------------------------
# plain forms


def _blocks(v, block):
    """[rows, cols] padded with zeros to whole blocks, as [rows / block, block, cols / 128, 128]."""
    rows, cols = v.shape
    v = torch.nn.functional.pad(v, (0, -cols % 128, 0, -rows % block))
    return v.view(v.shape[0] // block, block, v.shape[1] // 128, 128)


def _power(e):
    """2^e as float32, for whole e in [-127, 127], from its bits."""
    p = torch.bitwise_left_shift(e.to(torch.int32).clamp(min=-126) + 127, 23).view(torch.float32)
    return torch.where(e < -126, 0.5 * p, p)


def _quantize(x, block):
    """(values, scale bytes) of x's rows."""
    rows = x.shape[0]
    t = _blocks(x.float(), block)
    finite = torch.where(torch.isfinite(t), t.abs(), torch.zeros((), device=x.device))
    amax = finite.amax(dim=(1, 3), keepdim=True)
    # amax = f * 2^p with f in [0.5, 1), and 448 = 0.875 * 2^9
    f, p = torch.frexp(amax)
    e = torch.clamp(p - 9 + (f > 0.875), min=-127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    q = torch.where(torch.isfinite(t), t * _power(-e), torch.full((), math.nan, device=x.device))
    q = q.view(-1, q.shape[2] * 128)[:rows].to(FP8).contiguous()
    s = (e + 127).to(torch.uint8).view(e.shape[0], e.shape[2])
    return q, torch.nn.functional.pad(s, (0, -s.shape[1] % 4))


def _dequantize(q, s, block, k):
    scale = _power(s.to(torch.int32) - 127)[:, :q.shape[1] // 128]
    scale = scale.repeat_interleave(block, 0)[:q.shape[0]].repeat_interleave(128, 1)
    return (q.float() * scale)[:, :k]


def _statistics(x, kind):
    if kind == "rms":
        return None, torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    mean = x.mean(1, keepdim=True)
    return mean, torch.rsqrt(((x - mean) * (x - mean)).mean(1, keepdim=True) + EPS)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        out = []
        if s["form"] != "col":
            out += _quantize(s["x"], s["block"])
        if s["form"] != "row":
            out += _quantize(s["x"].t(), s["block"])
        return out
    if op == "matmul":
        a = _dequantize(s["a"], s["sa"], 1, s["k"])
        b = _dequantize(s["b"], s["sb"], s["block"], s["k"])
        return (a @ b.t()).to(TYPES[s["out"]])
    x = s["x"].float()
    if op == "norm":
        mean, rstd = _statistics(x, s["kind"])
        xhat = (x if mean is None else x - mean) * rstd
        y = xhat * s["weight"]
        y = y if s["b"] is None else y + s["b"]
        return [y.to(s["x"].dtype), rstd.view(-1)] + ([] if mean is None else [mean.view(-1)])
    dy, rstd = s["dy"].float(), s["rstd"].view(-1, 1)
    xhat = (x if s["mean"] is None else x - s["mean"].view(-1, 1)) * rstd
    g = dy * s["weight"]
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    dx = dx if s["mean"] is None else dx - g.mean(1, keepdim=True)
    return [(dx * rstd).to(s["x"].dtype), (dy * xhat).sum(0)] + ([dy.sum(0)] if s["bias"] else [])


def _own(s):
    import pretraining_optimizer_amd as pm
    op = s["op"]
    if op == "quantize":
        q = pm.fp8_quantize(s["x"], form=s["form"], block_rows=s["block"])
        return [t for m in (q if s["form"] == "both" else (q,)) for t in (m.data, m.scale)]
    if op == "matmul":
        return pm.fp8_matmul(pm.Fp8Matrix(s["a"], s["sa"], s["k"], 1), pm.Fp8Matrix(s["b"], s["sb"], s["k"], s["block"]),
                             out_dtype=TYPES[s["out"]])
    if op == "norm":
        y, mean, rstd = pm.norm_forward(s["x"], s["weight"], s["b"], kind=s["kind"], eps=EPS)
        return [y, rstd] + ([] if mean is None else [mean])
    dx, dweight, dbias = pm.norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], kind=s["kind"], bias=s["bias"])
    return [dx, dweight] + ([dbias] if s["bias"] else [])


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-k // 128)
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": (m + n) * k + (m + -(-n // case["block"])) * blocks + m * n * size, "flops": 2 * m * n * k}
    r, c = case["rows"], case["cols"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quantize":
        b = case["block"]
        row, col = r * c + -(-r // b) * -(-c // 128), r * c + -(-c // b) * -(-r // 128)
        return {"bytes": r * c * size + (row if case["form"] != "col" else 0) + (col if case["form"] != "row" else 0), "flops": 3 * r * c}
    stats = 4 * r * (2 if case["kind"] == "layer" else 1)
    vectors = 4 * c * (2 if case["bias"] else 1)
    if case["op"] == "norm":
        return {"bytes": 2 * r * c * size + stats + vectors, "flops": 6 * r * c}
    return {"bytes": 3 * r * c * size + stats + 4 * c + vectors, "flops": 12 * r * c}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _grid(v):
    """The nearest value with 4 significant bits and no exponent below -6 (ties to even), for |v| <= 448."""
    m, p = torch.frexp(v)
    step = torch.exp2(torch.clamp(p - 1, min=-6).double() - 3.0)
    return torch.round(v / step) * step


def _quantized(x, block):
    """_quantize's results from 64-bit logarithms and grids."""
    rows, cols = x.shape
    kb, rb = -(-cols // 128), -(-rows // block)
    full = torch.zeros((rb * block, kb * 128), dtype=torch.float64, device=x.device)
    full[:rows, :cols] = x.double()
    amax = full.abs().unfold(0, block, block).unfold(1, 128, 128).amax(dim=(2, 3))
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 448.0)) / 448.0)).clamp(min=-127)
    # a logarithm next to a whole number may round to either side of it
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where((amax > 0) & (amax <= 448.0 * torch.exp2(e - 1)) & (e > -127), e - 1, e)
    steps = torch.kron(torch.exp2(e), torch.ones((block, 128), dtype=torch.float64, device=x.device))
    s = torch.zeros((rb, -(-kb // 4) * 4), dtype=torch.float64, device=x.device)
    s[:, :kb] = e + 127
    return [_grid(full / steps)[:rows], s.to(torch.uint8)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        out = _quantized(s["x"], s["block"]) if s["form"] != "col" else []
        return out + (_quantized(s["x"].t().contiguous(), s["block"]) if s["form"] != "row" else [])
    if op == "matmul":
        def value(q, e, block):
            kb = q.shape[1] // 128
            steps = torch.pow(2.0, e[:, :kb].double() - 127.0)
            rows = torch.arange(q.shape[0], device=q.device) // block
            return (q.double().view(-1, kb, 128) * steps[rows].unsqueeze(2)).view(-1, kb * 128)
        return torch.matmul(value(s["a"], s["sa"], 1), value(s["b"], s["sb"], s["block"]).t().contiguous())
    x, w = s["x"].double(), s["weight"].double()
    n = x.shape[1]
    centre = x.sum(1) / n if s["kind"] == "layer" else None
    if op == "norm":
        d = x if centre is None else x - centre[:, None]
        r = 1.0 / torch.sqrt((d ** 2).sum(1) / n + EPS)
        y = d * r[:, None] * w[None, :]
        y = y if s["b"] is None else y + s["b"].double()[None, :]
        return [y, r] + ([] if centre is None else [centre])
    r, dy = s["rstd"].double()[:, None], s["dy"].double()
    h = (x if centre is None else x - s["mean"].double()[:, None]) * r
    p = dy * w[None, :]
    inner = (p * h).sum(1, keepdim=True) / n
    shift = p.sum(1, keepdim=True) / n if centre is not None else 0.0
    return [(p - shift - h * inner) * r, (dy * h).sum(0)] + ([dy.sum(0)] if s["bias"] else [])
