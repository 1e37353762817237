"""kv_cache_compact against the oracle's moves: bytes, equal everywhere, rows that nothing names among them."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
import oracle

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16}[t.element_size()])


def case(keys, block_size=16, Dv=512, Dk=64, dtype=torch.bfloat16, k_dtype=None, mode="PA_BSND", seed=0):
    g = torch.Generator().manual_seed(seed)
    n = len(keys)
    if mode == "Norm":
        d0, d1, table = n + 1, max(keys) + 2, None
    else:
        d1 = block_size
        pages = [-(-k // d1) for k in keys]
        d0 = sum(pages) + 3
        order = torch.randperm(d0, generator=g)
        table = torch.full((n, max(pages) + 1), -1, dtype=torch.int64)
        at = 0
        for i, p in enumerate(pages):
            table[i, :p] = order[at:at + p]
            at += p
    make = lambda w, t: bits(torch.empty(d0, d1, 1, w, dtype=t)).random_(0, 250, generator=g).view(t)  # noqa: E731
    return make(Dv, dtype), make(Dk, k_dtype or dtype), table


def run(c, kept, count, start=None, mode="PA_BSND", stream=None):
    ckv, k, table = c
    rv, rk = bits(ckv).numpy()[:, :, 0].copy(), bits(k).numpy()[:, :, 0].copy()
    rst = oracle.ref_kv_cache_compact(rv, rk, None if table is None else table.numpy(), kept, count, start)
    gv, gk, st = ckv.cuda(), k.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.kv_cache_compact(gv, gk, None if table is None else table.cuda(), torch.from_numpy(kept).cuda(), torch.tensor(count).cuda(),
                         start=None if start is None else torch.tensor(start).cuda(), cache_mode=mode, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == rst
    assert np.array_equal(bits(gv).cpu().numpy()[:, :, 0], rv) and np.array_equal(bits(gk).cpu().numpy()[:, :, 0], rk)
    return rst


def chosen(keys, counts, seed, start=None, most=None):
    """[N, most] ascending places of [start, keys), -1 behind the count."""
    r = np.random.default_rng(seed)
    out = np.full((len(keys), most or max(counts + [1])), -1, dtype=np.int64)
    for n, (K, m) in enumerate(zip(keys, counts)):
        s = start[n] if start else 0
        out[n, :m] = np.sort(r.choice(np.arange(s, K), m, replace=False))
    return out


@pytest.mark.parametrize("keys,counts,kw", [
    ([1], [1], {}), ([40], [17], {}), ([300, 1, 77, 500], [299, 0, 40, 1], dict(block_size=64)),
    ([5000], [4999], dict(block_size=128)), ([5000], [2500], dict(block_size=100)), ([3000, 2000, 1000], [1500, 1999, 10], dict(block_size=7)),
    ([4096] * 20, [2048] * 20, dict(block_size=128)), ([900] * 70, [450] * 70, {}), ([700, 333], [350, 111], dict(mode="Norm")),
    ([600, 90], [300, 45], dict(dtype=torch.float8_e4m3fn, k_dtype=torch.bfloat16)),
    ([600, 90], [300, 45], dict(dtype=torch.int8, k_dtype=torch.int8)),
    ([600, 90], [300, 45], dict(Dv=7, Dk=3, dtype=torch.int8)), ([3000], [1501], dict(Dv=70, Dk=6, dtype=torch.float16)),
    ([600, 90], [300, 45], dict(Dv=8, Dk=8)), ([2000], [1999], dict(Dv=8, Dk=8, dtype=torch.int8, k_dtype=torch.float16)),
    ([300, 44], [30, 40], dict(Dv=1024, Dk=256)), ([40000], [20000], dict(Dv=64, Dk=16, block_size=64))])
def test_kept_rows(keys, counts, kw):
    c = case(keys, seed=len(keys), **kw)
    assert run(c, chosen(keys, counts, 3), counts, mode=kw.get("mode", "PA_BSND")) == 0


@pytest.mark.parametrize("first", [1, 2, 700])
def test_rows_next_to_one_another(first):
    """All keys from `first` on move by `first`: every row that is written is read by another."""
    kept = np.arange(first, 5000, dtype=np.int64)[None]
    assert run(case([5000], 128, seed=first), kept, [5000 - first]) == 0


def test_accepted_branches():
    keys = [200 + 13 * n for n in range(90)]
    new = [9 + n % 23 for n in range(90)]
    counts = [n % 8 for n in range(90)]
    start = [a - b for a, b in zip(keys, new)]
    assert run(case(keys, 64, seed=4), chosen(keys, counts, 5, start), counts, start) == 0


def test_rows_that_stay():
    kept = np.array([[0, 1, 2, 3, 9, 11]])
    assert run(case([12], 4, seed=6), kept, [6]) == 0
    c = case([12], 4, seed=7)
    c[2][0, 0] = -1    # the block of the keys that stay need not be there
    assert run(c, kept, [6]) == 0


def test_what_is_refused_on_the_device():
    c = case([100, 50, 70], 16, seed=8)
    good = chosen([100, 50, 70], [30, 20, 10], 9)
    assert run(c, good, [30, 31, -1]) == 2
    assert run(c, good, [30, 20, 10], [0, 200, -5]) & 2
    bad = good.copy()
    bad[0, 29], bad[1, 19] = 10 ** 12, 7 * 16 + 100      # beyond the table
    assert run(c, bad, [30, 20, 10]) == 1
    below = np.array([[3, 9], [0, 1], [0, 1]])
    assert run(c, below, [2, 2, 2], [5, 0, 0]) == 1      # 3 < start
    same = np.array([[3, 3], [0, 1], [0, 1]])
    assert run(c, same, [2, 2, 2]) == 1
    table = c[2].clone()
    table[0, 5], table[1, 0], table[2, 4] = -1, 10 ** 9, -7
    assert run((c[0], c[1], table), good, [30, 20, 10]) == 1


def test_captured_and_on_another_stream():
    keys, counts = [900, 300], [400, 299]
    c, kept = case(keys, 64, seed=10), chosen([900, 300], [400, 299], 11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(c, kept, counts, stream=side)
    want = [c[0].cuda(), c[1].cuda()]
    got = [c[0].cuda(), c[1].cuda()]
    args = (c[2].cuda(), torch.from_numpy(kept).cuda(), torch.tensor(counts).cuda())
    kvr.kv_cache_compact(*want, *args)
    graph = torch.cuda.CUDAGraph()
    call = kvr.prepare_kv_cache_compact(*got, *args)
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(want[0]), bits(got[0])) and torch.equal(bits(want[1]), bits(got[1]))


def test_refusals():
    ckv, k, table = (x.cuda() for x in case([40, 40], 16, seed=1))
    i = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")  # noqa: E731
    for bad in ((ckv, k, None, i(2, 4), i(2)), (ckv, k, table, i(8), i(2)), (ckv, k, table, i(2, 4).int(), i(2)),
                (ckv, k, table, i(3, 4), i(3)), (ckv, k, table, i(2, 4), i(3)), (ckv, k[:2], table, i(2, 4), i(2)),
                (ckv.float(), k, table, i(2, 4), i(2))):
        with pytest.raises(ValueError):
            kvr.kv_cache_compact(*bad)
    with pytest.raises(ValueError):
        kvr.kv_cache_compact(ckv, k, table, i(2, 4), i(2), cache_mode="Norm")


def test_no_rotary_part():
    assert run(case([300, 44], 16, Dk=0, seed=12), chosen([300, 44], [100, 40], 13), [100, 40]) == 0
