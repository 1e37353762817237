"""mla_attention where the keys that exist change from step to step: holes in the block table at random, ragged ends, rows
in both CTAs of a pair and in several row tiles, every path that brings keys. The mask of a step is written by the warps
that bring its keys and read by the softmax warps; one of another step would show in every row."""
import numpy as np
import pytest

from attention_helpers import check_mla, mla_case, on_tensor_cores, oracle_mla, rounded_query, run_mla

pytestmark = pytest.mark.gpu

LAYOUTS = [(None, None), (None, "int8"), ("int8", None), ("fp8_e4m3fn", "fp8_e4m3fn")]   # latent, rotary part


def holes(keys, block_size, seed):
    r = np.random.default_rng(seed)
    return [(n, b) for n, k in enumerate(keys) for b in range(-(-k // block_size)) if r.random() < 0.4]


@pytest.mark.parametrize("cache,k_cache", LAYOUTS)
@pytest.mark.parametrize("block_size", [3, 8, 16, 32, 128])
def test_holes_everywhere(block_size, cache, k_cache):
    keys = [1700, 333, 64, 901, 30]
    c = mla_case([9, 1, 2, 30, 1], keys, 16, block_size=block_size, cache=cache, k_cache=k_cache,
                 holes=holes(keys, block_size, block_size), seed=50)
    assert on_tensor_cores(c)
    want = oracle_mla(c)
    got = [run_mla(c) for _ in range(3)]
    for g in got:
        check_mla(c, g, want)
        assert np.array_equal(g[0], got[0][0]) and np.array_equal(g[1], got[0][1])


@pytest.mark.parametrize("cache", [None, "int8"])
def test_ragged_ends(cache):
    """Sequences of 0 to 200 keys that end anywhere in a step, beside one another in a pair's work."""
    keys = [(n * 61) % 201 for n in range(90)]
    c = mla_case([1 + n % 3 for n in range(90)], keys, 40, cache=cache, scale_len=0, seed=51)
    q = rounded_query(c) if cache else [None, None]
    check_mla(c, run_mla(c), oracle_mla(c, *q))
