"""Random configurations of tree attention, key weights, selection and compaction against the oracle."""
import numpy as np
import pytest
import torch

from attention_helpers import check_mla, mla_case, on_tensor_cores, rounded_query
from cache_helpers import check_weight, oracle_tree, oracle_weight, row_lse, run_tree, run_weight, tree_words
import test_gpu_kv_compact as compact
import test_gpu_kv_select as select

pytestmark = pytest.mark.gpu


def step(r):
    """Arguments of mla_case."""
    n = int(r.integers(1, 7))
    new = [int(x) for x in r.integers(0, r.choice([2, 10, 70]), n)]
    new[0] = max(1, new[0])
    dtype = str(r.choice(["bf16", "f16"]))
    kw = dict(new=new, keys=[int(x) for x in r.integers(0, r.choice([40, 700]), n)], H=int(r.choice([1, 3, 8, 16, 40, 128])), dtype=dtype,
              block_size=int(r.choice([1, 7, 16, 32, 64, 100, 128])), mode=str(r.choice(["PA_BSND", "PA_BSND", "Norm"])),
              gap=int(r.integers(0, 3)), pad=int(r.choice([0, 0, 8])), seed=int(r.integers(1 << 30)))
    kw["Dv"], kw["Dk"] = [(512, 64), (512, 64), (256, 32), (128, 16), (80, 64), (33, 10)][int(r.integers(6))]
    if r.random() < 0.5:
        kw["cache"] = str(r.choice(["int8", "fp8_e4m3fn", "fp8_e5m2"]))
        kw["scale_len"] = int(r.choice([1, kw["Dv"]]))
        if r.random() < 0.4:
            kw["k_cache"], kw["k_scale_len"] = str(r.choice(["int8", "fp8_e4m3fn"])), int(r.choice([1, kw["Dk"]]))
    if kw["mode"] != "Norm":
        pages = [-(-k // kw["block_size"]) for k in kw["keys"]]
        kw["holes"] = [(i, int(r.integers(0, p))) for i, p in enumerate(pages) if p and r.random() < 0.3]
    return kw


@pytest.mark.parametrize("seed", range(40))
def test_key_weight(seed):
    r = np.random.default_rng(seed)
    c = mla_case(causal=bool(r.random() < 0.8), **step(r))
    lse, width = row_lse(c), max(1, int(c.key_length.max()) + int(r.integers(0, 4)))
    kw = dict(decay=float(r.choice([0.0, 0.5, 1.0]))) if r.random() < 0.6 else {}
    if kw:
        kw["past"] = torch.from_numpy(r.random((len(c.key_length), width)).astype(np.float32))
        kw["in_place"] = bool(r.random() < 0.5)
    gpu = run_weight(c, lse, width, pad=int(r.integers(0, 3)), **kw)
    check_weight(c, gpu, oracle_weight(c, lse, width, **kw), kw.get("past"), kw.get("decay", 1.0))


@pytest.mark.parametrize("seed", range(40))
def test_tree_attention(seed):
    r = np.random.default_rng(1000 + seed)
    c = mla_case(**step(r))
    mask = tree_words(c, -(-max(1, int((c.query_start[1:] - c.query_start[:-1]).max())) // 64) + int(r.integers(0, 2)), seed)
    q = rounded_query(c) if on_tensor_cores(c) else (None, None)
    check_mla(c, run_tree(c, mask), oracle_tree(c, mask, *q), p_rounded=on_tensor_cores(c))


@pytest.mark.parametrize("seed", range(25))
def test_select(seed):
    r = np.random.default_rng(2000 + seed)
    n, width = int(r.integers(1, 9)), int(r.choice([3, 40, 1000, 5000, 20000]))
    keep = int(r.integers(1, width + 2))
    sink = int(r.integers(0, min(keep, 9) + 1))
    kind = str(r.choice(["spread", "few", "equal", "odd"]))
    select.run(select.weights(n, width, seed, kind), [int(x) for x in r.integers(0, width + 1, n)], keep, sink,
               int(r.integers(0, keep - sink + 1)), pad=int(r.integers(0, 3)), carry=int(r.integers(0, 50)))


@pytest.mark.parametrize("seed", range(25))
def test_compact(seed):
    r = np.random.default_rng(3000 + seed)
    keys = [int(x) for x in r.integers(1, r.choice([30, 900, 3000]), int(r.integers(1, 20)))]
    start = [int(r.integers(0, k)) for k in keys] if r.random() < 0.5 else None
    counts = [int(r.integers(0, k - (start[i] if start else 0) + 1)) for i, k in enumerate(keys)]
    mode = str(r.choice(["PA_BSND", "PA_BSND", "Norm"]))
    types = [torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn]
    c = compact.case(keys, int(r.choice([1, 5, 16, 64, 128])), int(r.choice([512, 64, 33, 256])), int(r.choice([64, 8, 6])),
                     types[int(r.integers(4))], types[int(r.integers(4))], mode, seed)
    assert compact.run(c, compact.chosen(keys, counts, seed, start), counts, start, mode) == 0
