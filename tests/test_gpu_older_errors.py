"""A HIP call that failed earlier in the thread, here an allocation of a pebibyte
that the program gave up on, is not an error of the operators called after it."""

import ctypes

import pytest
import torch

import pretraining_optimizer_amd as pm
from parity import announce

pytestmark = pytest.mark.gpu


def _fail_an_allocation():
    # torch reports such an error itself where it takes new memory from HIP: leave
    # enough in its pools (one block above 1 MiB, some below) for the calls that follow
    spare = [torch.empty(1 << 28, dtype=torch.uint8, device="cuda")]
    spare += [torch.empty(1 << 19, dtype=torch.uint8, device="cuda") for _ in range(16)]
    del spare
    hip = ctypes.CDLL("libamdhip64.so")
    hip.hipMalloc.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_size_t]
    p = ctypes.c_void_p()
    assert hip.hipMalloc(ctypes.byref(p), 1 << 50) == 2   # hipErrorOutOfMemory


@pytest.fixture(autouse=True)
def _leave_no_error():
    yield
    ctypes.CDLL("libamdhip64.so").hipGetLastError()


def test_operators_after_a_failed_allocation():
    announce("operators after a failed allocation")
    x, w = torch.randn((401, 9000), device="cuda"), torch.randn((700, 9000), device="cuda")
    want_q = pm.fp8_quantize(x)
    q, qw = pm.Fp8Matrix.empty(401, 9000), pm.fp8_quantize(w)
    _fail_an_allocation()
    pm.fp8_quantize(x, out=q)
    assert torch.equal(q.data.view(torch.uint8), want_q.data.view(torch.uint8)) and torch.equal(q.scale, want_q.scale)
    # a split contraction: two launches
    want = pm.fp8_matmul(q, qw, out_dtype=torch.float32)
    c = torch.zeros((401, 700), device="cuda")
    torch.cuda.synchronize()
    _fail_an_allocation()
    pm.fp8_matmul(q, qw, out=c)
    assert torch.equal(c, want)
    gamma = torch.randn(9000, device="cuda")
    want = pm.norm_forward(x, gamma, kind="layer")
    wantg = pm.norm_backward(x, x, gamma, want[1], want[2], kind="layer", bias=True)
    _fail_an_allocation()
    got = pm.norm_forward(x, gamma, kind="layer")
    _fail_an_allocation()
    gotg = pm.norm_backward(x, x, gamma, got[1], got[2], kind="layer", bias=True)
    for a, b in zip(got + gotg, want + wantg):
        assert torch.equal(a, b)


@pytest.mark.parametrize("graph", [False, True])
def test_steps_after_a_failed_allocation(graph):
    announce(f"steps after a failed allocation, graph {graph}")
    w = torch.randn((300, 200), device="cuda")
    g = torch.randn((300, 200), device="cuda")
    ref, m, mr = w.clone(), torch.zeros_like(w), torch.zeros_like(w)
    a, b = pm.MuonH([w], [m], grad_dtype=torch.float32), pm.MuonH([ref], [mr], grad_dtype=torch.float32)
    forms = pm.fp8_quantize(w, form="both", block_rows=128)
    for k in range(3):
        torch.cuda.synchronize()
        _fail_an_allocation()
        if graph:
            a.step([g], elr=0.01, graph=True)
            b.step([g], elr=0.01, graph=True)
        else:
            a.step([g], elr=0.01, fp8=[forms])
            b.step([g], elr=0.01)
        assert torch.equal(w, ref) and torch.equal(m, mr), k
    if not graph:
        q, qt = pm.fp8_quantize(ref, form="both", block_rows=128)
        for x, y in zip(forms, (q, qt)):
            assert torch.equal(x.data.view(torch.uint8), y.data.view(torch.uint8)) and torch.equal(x.scale, y.scale)
    a.close()
    b.close()
