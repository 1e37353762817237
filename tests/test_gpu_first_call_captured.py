"""The first call of a process on a device may be one that a graph captures: looking up the kernels' limits and loading
them does not break the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
import attention_prologue_kv_gb300 as kvr
z = lambda *s: torch.randn(*s, device="cuda").bfloat16()
t = lambda *x: torch.tensor(x, device="cuda")
q, r, ckv, k, pos = z(2, 16, 512), z(2, 16, 64), z(4, 64, 1, 512), z(4, 64, 1, 64), t(3, 4)
args = (t(0, 2, 1, 3).view(1, 4), t(0, 2), t(200))
turned, out, rows, index = torch.zeros_like(r), torch.zeros_like(q), z(2, 576), t(5, 70)
def step():
    kvr.query_rope(r, pos, turned)
    kvr.mla_attention(q, turned, ckv, k, *args, out, softmax_scale=0.07)
    kvr.kv_cache_read(ckv, k, index, rows)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (turned, out, rows)]
for x in (turned, out, rows):
    x.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and float(b.float().abs().sum()) > 0 for a, b in zip(got, (turned, out, rows)))
"""


def test_a_captured_first_call():
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
