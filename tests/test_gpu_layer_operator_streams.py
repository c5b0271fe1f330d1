"""The attention, the residual norm and the embedding on a stream of their own, with
results that torch's current stream uses afterwards, and after a HIP call that
failed (MI355X only)."""

import ctypes

import pytest
import torch

import pretraining_optimizer_amd as pm
from parity import announce

pytestmark = pytest.mark.gpu

NAMES = ["attention", "attention_back", "add_norm", "add_norm_back", "embedding", "embedding_back"]


def _cases():
    """Calls of two inputs each, whose results are about as large: each gives its
    result's tensors."""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def make(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    q, do = make(2, 700, 8, 64), make(2, 700, 8, 64)
    k, v = make(2, 700, 2, 64), make(2, 700, 2, 64)
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    outs = [pm.attention_forward(q[i], k[i], v[i], cu) for i in (0, 1)]
    x, r, dy = make(2, 512, 1024), make(2, 512, 1024), make(2, 512, 1024)
    w = make(1024, dtype=torch.float32)
    stats = [pm.add_norm_quantize(x[i], r[i], w)[:2] for i in (0, 1)]
    tokens = torch.randint(0, 3000, (2, 9000), generator=gen, device="cuda")
    table, dout = make(3000, 256, dtype=torch.float32), make(2, 9000, 256)

    def norm(i, s):
        h, rstd, forms = pm.add_norm_quantize(x[i], r[i], w, form="both", stream=s)
        return [h, rstd] + [t for m in forms for t in (m.data.view(torch.uint8), m.scale)]

    return {
        "attention": lambda i, s: list(pm.attention_forward(q[i], k[i], v[i], cu, stream=s)),
        "attention_back": lambda i, s: list(pm.attention_backward(do[i], q[i], k[i], v[i], *outs[i], cu, stream=s)),
        "add_norm": norm,
        "add_norm_back": lambda i, s: list(pm.add_norm_backward(dy[i], x[1 - i], stats[i][0], w, stats[i][1], stream=s)),
        "embedding": lambda i, s: [pm.embedding_forward(tokens[i], table, scale=2.0, stream=s)],
        "embedding_back": lambda i, s: [pm.embedding_backward(tokens[i], dout[i], 3000, stream=s)],
    }


@pytest.mark.parametrize("name", NAMES)
def test_a_result_outlives_the_current_streams_use_of_it(name):
    """Dropped while the current stream has yet to read it, a result's memory is not
    given to the next call on its stream."""
    announce(f"results across streams: {name}")
    call = _cases()[name]
    s = torch.cuda.Stream()
    want = [[t.clone() for t in call(i, None)] for i in (0, 1)]
    torch.cuda.synchronize()
    first = call(0, s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(50_000_000)   # the current stream is behind
    kept = [t.clone() for t in first]
    at = {t.data_ptr() for t in first}
    del first
    second = call(1, s)
    assert not at & {t.data_ptr() for t in second}
    torch.cuda.synchronize()
    for a, b in zip(kept + second, want[0] + want[1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_calls_on_two_streams_at_once(name):
    """Each call has a workspace of its own."""
    announce(f"two streams: {name}")
    call = _cases()[name]
    want = [[t.clone() for t in call(i, None)] for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [call(k % 2, streams[k % 2]) for k in range(12)]
    torch.cuda.synchronize()
    for k, result in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(result, want[k % 2])), k


def _fail_an_allocation():
    # memory for the calls that follow, so that torch takes none from HIP
    spare = [torch.empty(1 << 28, dtype=torch.uint8, device="cuda")]
    spare += [torch.empty(1 << 19, dtype=torch.uint8, device="cuda") for _ in range(16)]
    del spare
    hip = ctypes.CDLL("libamdhip64.so")
    hip.hipMalloc.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_size_t]
    p = ctypes.c_void_p()
    assert hip.hipMalloc(ctypes.byref(p), 1 << 50) == 2   # hipErrorOutOfMemory


@pytest.mark.parametrize("name", NAMES)
def test_after_a_failed_allocation(name):
    """An error that an earlier call of the thread left behind is not the operator's."""
    announce(f"after a failed allocation: {name}")
    call = _cases()[name]
    want = call(0, None)
    torch.cuda.synchronize()
    try:
        _fail_an_allocation()
        got = call(0, None)
    finally:
        ctypes.CDLL("libamdhip64.so").hipGetLastError()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
