"""The device error word of the weight updates: calls whose first use is
inside a graph capture."""

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
