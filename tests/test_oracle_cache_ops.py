"""The oracle of drafted trees and bounded caches against closed forms and library routines."""
import numpy as np
import pytest

import oracle


def test_a_chain_sees_all_before_it():
    mask, pos = np.zeros((70, 2), dtype=np.int64), np.zeros(70, dtype=np.int64)
    assert oracle.ref_draft_tree(np.arange(70) - 1, [0, 70], mask, [5], pos) == 0
    bits = (mask.view(np.uint64)[:, :, None] >> np.arange(64, dtype=np.uint64) & np.uint64(1)).reshape(70, 128)[:, :70]
    assert np.array_equal(bits, np.tril(np.ones((70, 70), dtype=np.uint64)))
    assert np.array_equal(pos, 5 + np.arange(70))


def test_a_tree_by_hand():
    mask = np.full((6, 1), -9, dtype=np.int64)
    pos = np.full(6, -9, dtype=np.int64)
    assert oracle.ref_draft_tree([-1, 0, 0, 1, 9], [0, 4, 5], mask, [10, 20], pos) == 1   # the parent 9 does not come before
    assert mask[:, 0].tolist() == [1, 3, 5, 11, 1, -9] and pos.tolist() == [10, 11, 11, 12, 20, -9]
    assert oracle.ref_draft_tree([-1] * 65, [0, 65], np.zeros((65, 1), dtype=np.int64)) == 0x20


def attention_arrays(seed=0, T=5, H=2, keys=9):
    r = np.random.default_rng(seed)
    return (r.normal(size=(T, H, 8)), r.normal(size=(T, H, 4)), r.normal(size=(1, keys, 8)), r.normal(size=(1, keys, 4)))


def test_a_tree_that_is_a_chain_is_causal():
    qn, qr, ckv, k = attention_arrays()
    mask = np.zeros((5, 1), dtype=np.int64)
    oracle.ref_draft_tree(np.arange(5) - 1, [0, 5], mask)
    a, b = [(np.zeros((5, 2, 8)), np.zeros((5, 2))) for _ in range(2)]
    oracle.ref_mla_attention(qn, qr, ckv, k, None, [0, 5], [9], *a, scale=0.3)
    oracle.ref_mla_tree_attention(qn, qr, ckv, k, None, [0, 5], [9], mask, *b, scale=0.3)
    assert np.allclose(a[0], b[0], rtol=1e-13) and np.allclose(a[1], b[1], rtol=1e-13)


def test_weights_of_a_token_add_up_to_one():
    qn, qr, ckv, k = attention_arrays(1)
    out, lse = np.zeros((5, 2, 8)), np.zeros((5, 2))
    oracle.ref_mla_attention(qn, qr, ckv, k, None, [0, 5], [9], out, lse, scale=0.3)
    w = np.zeros((1, 9))
    oracle.ref_mla_key_weight(qn, qr, ckv, k, None, [0, 5], [9], lse, w, scale=0.3)
    assert np.isclose(w.sum(), 10.0, rtol=1e-13)
    again = w.copy()
    oracle.ref_mla_key_weight(qn, qr, ckv, k, None, [0, 5], [9], lse, again, scale=0.3, past=again, decay=0.5)
    assert np.allclose(again, 1.5 * w, rtol=1e-13)
    # the last key is seen by the last token alone
    p = np.exp(0.3 * (qn[4] @ ckv[0, 8] + qr[4] @ k[0, 8]) - lse[4]).sum()
    assert np.isclose(w[0, 8], p, rtol=1e-13)


@pytest.mark.parametrize("keep,sink,recent", [(4, 0, 0), (5, 2, 1), (3, 1, 2), (20, 3, 3)])
def test_select_against_argsort(keep, sink, recent):
    r = np.random.default_rng(keep)
    w = r.normal(size=(3, 12)).astype(np.float32)
    st, kept, count, carried = oracle.ref_kv_cache_select(w, [12, 7, 13], keep, sink, recent)
    assert st == 2 and count.tolist() == [min(12, keep), min(7, keep), 0] and (kept[2] == -1).all()
    for n, K in ((0, 12), (1, 7)):
        x = w[n, :K].astype(np.float64)
        x[:sink], x[K - recent:] = np.inf, np.inf
        want = np.sort(np.argsort(-x, kind="stable")[:keep])
        assert kept[n, :count[n]].tolist() == want.tolist() and np.array_equal(carried[n, :count[n]], w[n, want])


def test_select_ties_zeros_and_nan():
    w = np.array([[0.0, -0.0, 1.0, np.nan, 1.0, -np.inf]], dtype=np.float32)
    order = [3, 2, 4, 0, 1, 5]
    for keep in range(1, 6):
        assert oracle.ref_kv_cache_select(w, [6], keep)[1][0].tolist() == sorted(order[:keep])


def test_compact_is_one_assignment():
    r = np.random.default_rng(3)
    ckv, k = r.normal(size=(4, 5, 3)), r.normal(size=(4, 5, 2))
    table = np.array([[2, 0, 3]])
    flat = lambda x: x[table[0]].reshape(15, -1)  # noqa: E731
    a, b = flat(ckv).copy(), flat(k).copy()
    kept = np.array([[2, 4, 7, 11, -1]])
    assert oracle.ref_kv_cache_compact(ckv, k, table, kept, [4], [2]) == 0
    a[[2, 3, 4, 5]], b[[2, 3, 4, 5]] = a[[2, 4, 7, 11]], b[[2, 4, 7, 11]]
    assert np.array_equal(flat(ckv), a) and np.array_equal(flat(k), b)
    assert oracle.ref_kv_cache_compact(ckv, k, table, np.array([[3, 3]]), [2]) == 1
    assert oracle.ref_kv_cache_compact(ckv, k, table, kept, [6]) == 2
