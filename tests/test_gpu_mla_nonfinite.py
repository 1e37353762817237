"""mla_attention with NaN and infinities in queries and in keys that are used, on the tensor-core kernel (512 + 64
channels) and on the plain one (10 + 6): what the definition makes NaN is NaN, what it leaves finite keeps its bits."""
import copy

import numpy as np
import pytest

from attention_helpers import mla_case, on_tensor_cores, run_mla

pytestmark = pytest.mark.gpu

NEW, KEYS, H = [3, 1], [150, 40], 5


def case(Dv, Dk, dtype="bf16", cache=None, new=NEW, keys=KEYS):
    c = mla_case(new, keys, H, Dv, Dk, dtype=dtype, cache=cache, seed=40)
    assert on_tensor_cores(c) == (Dv == 512)
    return c


def spoiled(c, part, rows, value):
    """The case with `value` in the last channel of `part` of the query rows (token, head)."""
    d = copy.copy(c)
    d.q_nope, d.q_rope = c.q_nope.clone(), c.q_rope.clone()   # tensors of their own, which run_mla takes as they are
    for t, h in rows:
        getattr(d, part)[t, h, -1] = value
    return d


@pytest.mark.parametrize("part", ["q_nope", "q_rope"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("Dv,Dk", [(512, 64), (10, 6)])
@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("f16", None), ("bf16", "int8"), ("f16", "fp8_e4m3fn")])
def test_a_query_row_that_is_not_finite(part, value, Dv, Dk, dtype, cache):
    """Some of an infinite query's scores are +inf, so that its softmax is NaN as a NaN query's is."""
    c = case(Dv, Dk, dtype, cache)
    rows = [(0, 2), (2, 0), (3, 4)]
    want, got = run_mla(c), run_mla(spoiled(c, part, rows, value))
    at = np.zeros(want[1].shape, bool)
    for t, h in rows:
        at[t, h] = True
    assert np.isnan(got[0][at]).all() and not np.isfinite(got[1][at]).any()
    if np.isnan(value):
        assert np.isnan(got[1][at]).all()
    assert np.array_equal(got[0][~at], want[0][~at]) and np.array_equal(got[1][~at], want[1][~at])
    assert got[2] == 0


@pytest.mark.parametrize("Dv,Dk", [(512, 64), (10, 6)])
def test_a_nan_query_that_sees_no_key_or_one(Dv, Dk):
    """Zeros where nothing is seen, whatever the query; NaN from the first key on."""
    c = case(Dv, Dk, new=[2, 1], keys=[1, 0])
    got = run_mla(spoiled(c, "q_nope", [(0, 1), (1, 1), (2, 1)], float("nan")))
    assert (got[0][[0, 2]] == 0).all() and np.isneginf(got[1][[0, 2]]).all()
    assert np.isnan(got[0][1, 1]).all() and np.isnan(got[1][1, 1])
    assert np.isfinite(got[0][1, 0]).all() and np.isfinite(got[1][1, 0])


@pytest.mark.parametrize("Dv,Dk", [(512, 64), (10, 6)])
def test_scores_of_minus_infinity(Dv, Dk):
    """An infinite query over keys of one sign: every score is -inf, and the row as one that sees no key."""
    c = case(Dv, Dk)
    for t in (c.ckv, c.k):
        t.view(-1, t.shape[-1])[:, -1] = t.view(-1, t.shape[-1])[:, -1].abs() + 0.5
    want = run_mla(c)
    got = run_mla(spoiled(c, "q_rope", [(1, 3)], float("-inf")))
    assert (got[0][1, 3] == 0).all() and np.isneginf(got[1][1, 3])
    rest = np.ones(want[1].shape, bool)
    rest[1, 3] = False
    assert np.array_equal(got[0][rest], want[0][rest]) and np.array_equal(got[1][rest], want[1][rest])


@pytest.mark.parametrize("key", [0, 63, 149])
@pytest.mark.parametrize("part", ["ckv", "k"])
@pytest.mark.parametrize("Dv,Dk,cache", [(512, 64, None), (512, 64, "fp8_e4m3fn"), (10, 6, None), (10, 6, "fp8_e4m3fn")])
def test_a_nan_key_reaches_the_tokens_that_see_it_and_no_other_sequence(key, part, Dv, Dk, cache):
    c = case(Dv, Dk, cache=cache)
    want = run_mla(c)
    d = copy.copy(c)
    t = getattr(c, part).clone()
    t.view(-1, t.shape[-1])[c.table[0, key // 16] * 16 + key % 16] = float("nan")
    setattr(d, part, t)
    got = run_mla(d)
    sees = [j for j in range(3) if key < 150 - 3 + j + 1]
    assert np.isnan(got[0][sees]).all() and np.isnan(got[1][sees]).all()
    assert np.array_equal(got[0][3], want[0][3]) and np.array_equal(got[1][3], want[1][3])
