"""The device error word of the weight updates: calls whose first use is
inside a graph capture, and what a call leaves behind when a device wait ran
out of time (marked from the host: no wait really runs out)."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALL_IN_A_CAPTURE = """
import torch
from mixture_experts_routed_route_gb300 import optim
g = torch.randn(2, 96, 160, device="cuda")
out = torch.empty(2, 96, 160, device="cuda", dtype=torch.bfloat16)
junk = torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda")   # what a new allocation may hold
del junk
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    optim.orthogonalize(g, out=out)
for _ in range(2):
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, optim.orthogonalize(g))
    assert optim.error_bits() == 0
print("first call captured")
"""


def test_first_call_of_a_process_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stderr[-2000:]


@pytest.fixture
def lost_product():
    """Sets the product that counts as lost; none after the test."""
    from mixture_experts_routed_route_gb300 import abi
    yield abi.moe_test_muon_lost
    abi.moe_test_muon_lost(-1)


@pytest.mark.parametrize("E,N,K,matrices", [(3, 300, 520, 3), (3, 520, 300, 2), (5, 300, 281, 2), (1, 256, 4096, 1)])
def test_weights_stay_when_a_product_is_lost(lost_product, E, N, K, matrices):
    from test_gpu_muon import gradient

    from mixture_experts_routed_route_gb300 import abi, optim
    ws = optim.workspace(E, N, K, matrices=matrices)
    grad = gradient(E, N, K).bfloat16()
    good = optim.orthogonalize(grad, workspace=ws)
    for product in (0, 1, 2, 7, 13):
        for dtype in (torch.float32, torch.bfloat16):
            w = torch.randn((E, N, K), device="cuda").to(dtype)
            m = torch.ones((E, N, K), device="cuda")
            c = torch.zeros((E, N, K), device="cuda", dtype=torch.bfloat16) if dtype is torch.float32 else None
            w0 = w.clone()
            lost_product(product)
            optim.muon_update(w, grad, m, lr=0.1, mu=0.5, weight_bf16=c, workspace=ws)
            out = torch.full_like(good, 7.0)
            optim.orthogonalize(grad, out=out, workspace=ws)
            lost_product(-1)
            assert optim.error_bits() == abi.MOE_DEV_ERR_TIMEOUT
            assert torch.equal(w, w0) and (c is None or float(c.abs().max()) == 0.0)
            assert bool((out == 7.0).all())
            assert torch.equal(m, 0.5 + grad.float())
            # the next call finds nothing of it
            assert torch.equal(optim.orthogonalize(grad, workspace=ws), good)
            assert optim.error_bits() == 0
            optim.muon_update(w, grad, m, lr=0.1, mu=0.5, weight_bf16=c, workspace=ws)
            assert not torch.equal(w, w0) and optim.error_bits() == 0
