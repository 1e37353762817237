"""The first calls of a process on the operators of a bounded cache may be ones that a graph captures."""
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
i = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")
q, r, ckv, k = z(3, 16, 512), z(3, 16, 64), z(4, 64, 1, 512), z(4, 64, 1, 64)
table, start, length = t(0, 2, 1, 3).view(1, 4), t(0, 3), t(200)
codes, scale = (z(4, 64, 1, 512) * 20).to(torch.int8), torch.full((1,), 20.0, device="cuda")
mask, out, lse = i(3, 1), torch.zeros_like(q), torch.zeros(3, 16, device="cuda")
w, w8 = torch.zeros(1, 256, device="cuda"), torch.zeros(1, 256, device="cuda")
kept, count, long, far = i(1, 100), i(1), torch.rand(1, 200000, device="cuda"), i(1, 1000)
held = (ckv.clone(), k.clone())
def step():
    ckv.copy_(held[0])
    k.copy_(held[1])
    kvr.draft_tree(t0, start, mask)
    kvr.mla_attention(q, r, ckv, k, table, start, length, out, softmax_scale=0.07, lse=lse, tree_mask=mask)
    kvr.mla_key_weight(q, r, ckv, k, table, start, length, lse, w, softmax_scale=0.07)
    kvr.mla_key_weight(q, r, codes, k, table, start, length, lse, w8, softmax_scale=0.07, ckv_scale=scale)
    kvr.kv_cache_select(w, length, kept, count, sink=2, recent=8)
    kvr.kv_cache_compact(ckv, k, table, kept, count)
    kvr.kv_cache_select(long, full, far, count)
t0, full = t(-1, 0, 0), t(200000)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
outs = (mask, out, lse, w, w8, kept, ckv, k, far)
got = [x.clone() for x in outs]
for x in outs:
    x.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and float(b.float().abs().sum()) > 0 for a, b in zip(got, outs))
"""


def test_captured_first_calls():
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
