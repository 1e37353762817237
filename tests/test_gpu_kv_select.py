"""kv_cache_select against sorting: whole numbers and carried weights, equal everywhere."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
import oracle
from helpers import guarded

pytestmark = pytest.mark.gpu


def run(w, length, keep, sink=0, recent=0, pad=0, carry=0, stream=None):
    n, width = w.shape
    rst, rk, rc, rw = oracle.ref_kv_cache_select(w, length, keep, sink, recent)
    wide = torch.zeros(n, width + pad)
    wide[:, :width] = torch.from_numpy(w)
    kept, c1 = guarded((n, keep), torch.int64, -5)
    count, c2 = guarded((n,), torch.int64, -5)
    carried, c3 = guarded((n, keep + carry), torch.float32, -5.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.kv_cache_select(wide.cuda()[:, :width], torch.tensor(length, dtype=torch.int64).cuda(), kept, count, sink=sink, recent=recent,
                        kept_weight=carried, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    for check in (c1, c2, c3):
        check()
    assert int(st.item()) == rst
    assert np.array_equal(count.cpu().numpy(), rc)
    assert np.array_equal(kept.cpu().numpy(), rk)
    got = carried.cpu().numpy()
    assert np.array_equal(got[:, :keep].view(np.int32), rw.view(np.int32)) and (got[:, keep:] == 0).all()


def weights(n, width, seed, kind="spread"):
    r = np.random.default_rng(seed)
    if kind == "equal":
        return np.full((n, width), 0.5, dtype=np.float32)
    if kind == "few":
        return r.integers(0, 5, (n, width)).astype(np.float32) / 4 - 0.5
    if kind == "odd":
        x = r.normal(size=(n, width)).astype(np.float32)
        x[r.random((n, width)) < 0.2] = np.nan
        x[r.random((n, width)) < 0.1] = np.inf
        x[r.random((n, width)) < 0.1] = -np.inf
        x[r.random((n, width)) < 0.1] = -0.0
        x[r.random((n, width)) < 0.1] = 0.0
        x[r.random((n, width)) < 0.1] = 1e-42
        return x
    return np.exp(2 * r.normal(size=(n, width))).astype(np.float32)


@pytest.mark.parametrize("kind", ["spread", "few", "equal", "odd"])
@pytest.mark.parametrize("n,width,keep,sink,recent", [
    (1, 1, 1, 0, 0), (1, 33, 32, 0, 0), (3, 700, 100, 4, 32), (5, 2049, 1, 0, 1), (2, 4097, 4096, 1, 1), (2, 4097, 2048, 2048, 0),
    (2, 4000, 1500, 0, 1500), (40, 513, 200, 3, 9), (1, 20011, 5000, 4, 512), (2, 9000, 9000, 1, 1), (2, 900, 2000, 5, 7)])
def test_sizes(kind, n, width, keep, sink, recent):
    r = np.random.default_rng(width)
    length = [int(x) for x in r.integers(width // 2, width + 1, n)]
    length[0] = width
    run(weights(n, width, keep, kind), length, keep, sink, recent, carry=7)


def test_lengths():
    w = weights(6, 3000, 1)
    run(w, [0, 1, 500, 501, 3000, 2999], 500, 3, 10, pad=5, carry=100)
    run(w, [-1, 1, 3001, 501, -(1 << 60), 1 << 60], 500, 3, 10)


@pytest.mark.parametrize("width", [131072, 400001, 700003])
def test_one_long_sequence(width):
    """Shares of eight CTAs that fit their shared memory, the last one's beyond it."""
    run(weights(1, width, 3), [width - 5], width // 4, 4, 512)
    run(weights(1, width, 4, "few"), [width], width // 3, 0, 0)


def test_keys_that_are_read_again():
    """More than registers and shared memory of sixteen CTAs hold."""
    run(weights(1, 900001, 7), [900001], 3000, 4, 512)
    run(weights(2, 900001, 8, "odd"), [900000, 850000], 400000, 4, 512, pad=1)


@pytest.mark.parametrize("least", [-1.01, -2.0, -3.7, -1e30, -np.inf])
def test_ranges_up_to_the_last_rank(least):
    """NaN, the highest rank, above a negative least weight: the bin that ends the range reaches beyond 32 bits."""
    w = np.array([[least] + [np.nan] * 5 + [1.0, 2.0, 1.0, 0.5, -0.25, np.inf, 3.0]], dtype=np.float32)
    for keep in range(1, 13):
        run(w, [13], keep)


def test_many_sequences():
    run(weights(1000, 40, 5, "few"), [int(x) for x in np.random.default_rng(1).integers(0, 41, 1000)], 16, 2, 3)


def test_captured_and_on_another_stream():
    w = torch.from_numpy(weights(4, 3000, 6)).cuda()
    length = torch.tensor([3000, 10, 2000, 700]).cuda()
    outs = [(torch.zeros(4, 600, dtype=torch.int64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")) for _ in range(3)]
    kvr.kv_cache_select(w, length, *outs[0], sink=4, recent=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kvr.kv_cache_select(w, length, *outs[1], sink=4, recent=9, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvr.kv_cache_select(w, length, *outs[2], sink=4, recent=9)
    graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])


def test_refusals():
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")  # noqa: E731
    for bad in ((z(2, 9).double(), i(2), i(2, 4), i(2)), (z(2, 9), i(3), i(2, 4), i(2)), (z(2, 9), i(2), i(3, 4), i(2)),
                (z(2, 9), i(2).int(), i(2, 4), i(2)), (z(1, 9).expand(2, 9), i(2), i(2, 4), i(2)), (z(2, 9), i(2), i(8), i(2))):
        with pytest.raises(ValueError):
            kvr.kv_cache_select(*bad)
    for kw in (dict(sink=3, recent=2), dict(sink=-1), dict(kept_weight=z(2, 3))):
        with pytest.raises(kvr.KvrError):
            kvr.kv_cache_select(z(2, 9), i(2), i(2, 4), i(2), **kw)
