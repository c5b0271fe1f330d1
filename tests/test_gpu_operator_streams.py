"""Results of operators that ran on a stream of their own and are used on torch's
current stream afterwards (MI355X only)."""

import pytest
import torch

import pretraining_optimizer_amd as pm
from parity import announce

pytestmark = pytest.mark.gpu


def _cases():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, 512, 1024), generator=gen, device="cuda")
    w = torch.randn(1024, generator=gen, device="cuda")
    q = [pm.fp8_quantize(t) for t in x]
    stats = [pm.norm_forward(t, w, kind="layer") for t in x]
    return {
        "quantize": lambda i, s: [pm.fp8_quantize(x[i], stream=s).data.view(torch.uint8)],
        "matmul": lambda i, s: [pm.fp8_matmul(q[i], q[0], stream=s)],
        "norm": lambda i, s: [t for t in pm.norm_forward(x[i], w, kind="layer", stream=s)],
        "norm_back": lambda i, s: list(pm.norm_backward(x[i], x[1 - i], w, *stats[1 - i][1:], kind="layer", bias=True, stream=s)),
    }


@pytest.mark.parametrize("name", ["quantize", "matmul", "norm", "norm_back"])
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
    # read and done: the memory is used again
    del second
    third = call(0, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(third, want[0]))
