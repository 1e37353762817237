"""draft_tree against the oracle: whole numbers, equal everywhere."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
import oracle
from cache_helpers import parents

pytestmark = pytest.mark.gpu


def run(parent, start, words, T=None, first=None, want_positions=True, shared=()):
    """shared: rows of two sequences, the first of which the oracle's result does not show."""
    T = len(parent) if T is None else T
    up = torch.full((T,), -1, dtype=torch.int64)
    up[:len(parent)] = torch.as_tensor(parent)
    mask, pos = torch.full((T, words), -9, dtype=torch.int64), torch.full((T,), -9, dtype=torch.int64)
    rm, rp = mask.numpy().copy(), pos.numpy().copy()
    rst = oracle.ref_draft_tree(up.numpy(), start, rm, first, rp if want_positions else None)
    gm, gp, st = mask.cuda(), pos.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.draft_tree(up.cuda(), torch.tensor(start).cuda(), gm, position_start=torch.tensor(first).cuda() if want_positions else None,
                   positions=gp if want_positions else None, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == rst
    gm, gp = gm.cpu().numpy(), gp.cpu().numpy()
    if len(shared):   # either sequence's words and position
        assert start[2] < start[1]
        lm, lp = np.zeros_like(rm), np.zeros_like(rp)
        oracle.ref_draft_tree(up.numpy(), start[:2], lm, first, lp)
        for t in shared:
            assert gm[t] in (rm[t], lm[t]) and gp[t] in (rp[t], lp[t])
            gm[t], gp[t] = rm[t], rp[t]
    assert np.array_equal(gm, rm) and np.array_equal(gp, rp)


@pytest.mark.parametrize("counts,words,chain", [
    ([1], 1, False), ([26], 1, False), ([64], 1, True), ([65], 2, True), ([128, 127, 1, 0, 129], 3, False), ([4096], 64, True),
    ([4095, 1], 64, False), ([5] * 700, 1, False), ([200, 33], 8, False)])
def test_trees(counts, words, chain):
    start = np.concatenate([[0], np.cumsum(counts)]).tolist()
    first = [(7919 * n) % 100003 - 50 for n in range(len(counts))]
    run(parents(counts, sum(counts), chain), start, words, first=first)
    run(parents(counts, sum(counts) + 1, chain), start, words, T=sum(counts) + 3, first=first)   # rows behind the last sequence
    run(parents(counts, sum(counts) + 2, chain), start, words, want_positions=False)


def test_more_sequences_than_ctas():
    counts = [1, 2, 3] * 1700
    run(parents(counts, 1), np.concatenate([[0], np.cumsum(counts)]).tolist(), 1, first=list(range(len(counts))))


def test_bad_parents_and_sequences():
    run([-1, 0, 2, 1, -2, 4, 1 << 40, -(1 << 63)], [0, 8], 1, first=[3])
    run([-1] * 70, [0, 65, 70], 1, first=[1, 2])                      # 65 tokens, one word
    run([-1, 0, 1, 2, 3, 0], [0, 4, 2, 6], 1, first=[1, 2, 3], shared=[2, 3])   # query_start decreases
    run([-1, 0, 1], [0, 2, 5], 1, first=[1, 2])                       # it leaves [0, T]
    run([-1, 0, 1], [-1, 2, 3], 1, first=[1, 2])
