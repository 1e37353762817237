"""mla_attention with a tree mask against the float64 oracle."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
from attention_helpers import check_mla, mla_case, on_tensor_cores, rounded_query, run_mla
from cache_helpers import cuda, oracle_tree, queries, run_tree, tree_words
from helpers import f64

pytestmark = pytest.mark.gpu


def check(c, mask, rounded=False):
    gpu = run_tree(c, mask)
    q = rounded_query(c) if rounded else (None, None)
    check_mla(c, gpu, oracle_tree(c, mask, *q), p_rounded=on_tensor_cores(c))
    return gpu


@pytest.mark.parametrize("kw", [
    dict(new=[1], keys=[1], H=16),
    dict(new=[26], keys=[1026], H=16),
    dict(new=[7, 1, 64, 33], keys=[500, 1, 64, 90], H=20, block_size=64),
    dict(new=[31, 8], keys=[31, 70], H=128, block_size=128),
    dict(new=[65, 130], keys=[700, 130], H=8, block_size=32),
    dict(new=[17, 3], keys=[129, 40], H=24, dtype="f16", block_size=100),
    dict(new=[40], keys=[300], H=5, block_size=1),
    dict(new=[19, 2, 50], keys=[400, 33, 91], H=12, mode="Norm"),
    dict(new=[12, 30], keys=[200, 180], H=16, cache="int8", dtype="f16"),
    dict(new=[12, 30], keys=[200, 180], H=16, cache="fp8_e5m2"),
    dict(new=[21], keys=[333], H=32, Dv=256, Dk=32, pad=8, block_size=64),
    dict(new=[9, 14], keys=[77, 130], H=3, Dv=70, Dk=6),
    dict(new=[9, 14], keys=[77, 130], H=3, Dv=600, Dk=64, dtype="f16")])
def test_random_trees(kw):
    c = mla_case(seed=len(kw["new"]) + kw.get("H", 4), **kw)
    check(c, tree_words(c, -(-max(kw["new"]) // 64), 5))


@pytest.mark.parametrize("kw", [dict(cache="fp8_e4m3fn", scale_len=512), dict(cache="int8", scale_len=512, dtype="f16")])
def test_scales_per_channel(kw):
    c = mla_case([13, 40], [300, 90], H=16, block_size=64, seed=4, **kw)
    check(c, tree_words(c, 1, 6), rounded=True)


def test_a_chain_is_causal():
    """The same tokens as a chain of drafted ones and causally: equal to the last bit."""
    for kw in (dict(new=[30, 1, 64], keys=[500, 20, 64], H=16, block_size=64), dict(new=[5, 9], keys=[70, 9], H=3, Dv=72, Dk=10)):
        c = mla_case(seed=9, **kw)
        a, b = run_mla(c), run_tree(c, tree_words(c, 1, 1, chain=True))
        if on_tensor_cores(c):   # the work is cut elsewhere
            assert np.abs(a[0] - b[0]).max() <= 2.0 ** -7 * np.abs(a[0]).max()
        else:
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_rows_that_see_nothing_and_bits_behind_the_last_token():
    c = mla_case([6, 40, 3], [6, 100, 50], H=16, seed=3, gap=4)
    mask = tree_words(c, 2, 8)
    mask[0:6] = 0        # no context and no ancestor: zeros, lse -inf
    mask[2, 0] = -1      # bits behind its 6 tokens name no key
    mask[7, 0] = 1 << 39
    mask[8, 1] = -1
    gpu = check(c, mask)
    assert (gpu[0][0] == 0).all() and np.isneginf(gpu[1][0]).all()
    assert (gpu[0][-4:] == -77).all()


def test_more_new_tokens_than_keys():
    c = mla_case([50, 20], [30, 5], H=8, seed=5)
    check(c, tree_words(c, 1, 2))


def test_holes_and_too_many_tokens():
    c = mla_case([20, 65, 4], [300, 200, 77], H=8, block_size=16, seed=6, holes=[(0, 2), (0, 18), (2, 4)])
    mask = tree_words(c, 2, 3)
    check(c, mask)
    one = mask[:, :1].contiguous()   # the second sequence's 65 tokens do not fit: left out
    gpu = check(c, one)
    assert gpu[2] == 0x20 and (gpu[0][20:85] == -77).all()


@pytest.mark.parametrize("H", [16, 128])
def test_long_contexts_cut_over_many_ctas(H):
    c = mla_case([26, 9], [5000, 3001], H=H, block_size=128, seed=7)
    check(c, tree_words(c, 1, 4))


def test_captured_replayed_and_on_another_stream():
    c = mla_case([26, 9], [700, 301], H=16, block_size=64, seed=8)
    mask = tree_words(c, 1, 5)
    want = run_tree(c, mask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run_tree(c, mask, stream=side)
    assert np.array_equal(want[0], again[0]) and np.array_equal(want[1], again[1])
    out = torch.zeros(c.q_nope.shape, dtype=c.q_nope.dtype, device="cuda")
    words = mask.cuda()
    call = kvr.prepare_mla_attention(*queries(c), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length), out,
                                     softmax_scale=c.scale, tree_mask=words)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(f64(out), want[0])
    words.copy_(tree_words(c, 1, 6))   # another tree at the same place
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(f64(out), run_tree(c, words.cpu())[0])


def test_refusals():
    c = mla_case([3], [20], H=4, seed=1)
    good = tree_words(c, 1, 1)
    for bad in (good.int(), good[:2], good[:, 0], good.t().contiguous(), torch.zeros(3, 0, dtype=torch.int64)):
        with pytest.raises(ValueError):
            run_tree(c, bad)
    with pytest.raises(ValueError):
        kvr.mla_attention(*queries(c), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length),
                          torch.zeros_like(c.q_nope, device="cuda"), softmax_scale=1.0, tree_mask=good)
