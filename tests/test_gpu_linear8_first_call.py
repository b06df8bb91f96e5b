"""The first call of each kernel of a process inside a graph's capture: what a launch asks of the runtime is allowed there."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import block_scaled_quantized_tcgen05_gb300 as q
q.qgemm_poll_device_error()                     # the library's own memory
def product(m, n, k):
    a, w = (torch.randint(-127, 128, s, dtype=torch.int8, device="cuda") for s in ((m, k), (n, k)))
    sa, sw, c = torch.ones(m, device="cuda"), torch.ones(n, device="cuda"), torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    return c, lambda: q.qgemm_w8a8(a, sa, w, sw, c)
def rows(t, h, up):
    x = torch.randn(t, h, device="cuda").half()
    y, s = torch.zeros(t, h, dtype=torch.int8, device="cuda"), torch.zeros(t, device="cuda")
    if up:
        return y, lambda: q.qgemm_act_quant(x, y, s, up=x, activation="silu")
    return y, lambda: q.qgemm_norm_quant(x, None, y, s)
calls = [product(*s) for s in ((8, 512, 8192), (16, 4096, 1024), (30, 1024, 4096), (48, 1024, 1024), (48, 4096, 1024), (200, 512, 4096),
                               (700, 2048, 512))]
calls += [rows(*s) for s in ((300, 4096, False), (5, 14336, False), (300, 28672, True), (300, 100, False), (9, 40000, True))]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for _, call in calls:
        call()
graph.replay()
torch.cuda.synchronize()
captured = [out.clone() for out, _ in calls]
for (out, call), first in zip(calls, captured):
    out.zero_()
    call()
    assert torch.equal(out, first) and bool(first.any())
assert q.qgemm_poll_device_error() == 0
print("same")
"""


def test_first_calls_captured():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
