"""How exact mla_key_weight's weights are, against the float64 oracle: the root mean square of their relative errors.

Bound, for N(0, 1) queries and values at a scale of 0.0722 and few rows, so that errors do not average out. A score is 36 additions
of 16 products (twice as many where queries are held in two parts), each cut off by 2^-23 of the sum so far at most, 2^-24 in the
mean, and that sum is 24 in the mean square: 0.0722 x 36 x 2^-24 x 24 = 3.7e-6 of a weight, 7.4e-6 with two parts. The exponent adds
the roundings of lse log2 e, of the score's factor and of their difference, 3 x 2^-24 x 12 = 2.1e-6, and the exponential 2^-22. Parts
of 22 bits add 2^-23 x 0.0722 x 24 = 2e-7, two parts in bf16 of the rotary 64 channels 2^-17 / sqrt(3) x 0.0722 x 8 = 2.5e-6. Together
less than 1e-5 for caches of 16 bits and 1.5e-5 for codes."""
import numpy as np
import pytest
import torch

from attention_helpers import DTYPES, mla_case
from cache_helpers import oracle_weight, row_lse, run_weight

CODES = [(dtype, cache, scale_len, k_cache) for dtype in ("bf16", "f16")
         for cache, k_cache in (("int8", None), ("fp8_e4m3fn", None), ("fp8_e5m2", None), ("fp8_e4m3fn", "fp8_e4m3fn"))
         for scale_len in (1, 512)]
LIMIT16, LIMIT8 = 1e-5, 1.5e-5


def case(dtype, cache=None, scale_len=1, k_cache=None, **kw):
    return mla_case([1, 1, 2], [900, 300, 513], H=2, dtype=dtype, cache=cache, scale_len=scale_len, k_cache=k_cache,
                    seed=41, **dict(dict(block_size=64), **kw))


def rms(w, ref):
    at = (ref > 0) & (ref != -77.0)
    return float(np.sqrt(np.mean(((w[at] - ref[at]) / ref[at]) ** 2)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kw", [dict(), dict(block_size=100), dict(Dv=256, Dk=32)])
def test_caches_of_16_bits(dtype, kw):
    c = case(dtype, **kw)
    lse = row_lse(c)
    assert rms(run_weight(c, lse, 900)[0], oracle_weight(c, lse, 900)[0]) < LIMIT16


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache,scale_len,k_cache", CODES)
def test_caches_of_codes(dtype, cache, scale_len, k_cache):
    c = case(dtype, cache, scale_len, k_cache)
    lse = row_lse(c)
    assert rms(run_weight(c, lse, 900)[0], oracle_weight(c, lse, 900)[0]) < LIMIT8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache,scale_len,k_cache", CODES)
def test_scores_of_the_rotary_part_alone(dtype, cache, scale_len, k_cache):
    """Latent queries of zero: 64 channels carry the score, a third of its size in the mean square, at three times the scale."""
    c = case(dtype, cache, scale_len, k_cache, scale=0.0722 * 3)
    c.q_nope.zero_()
    lse = row_lse(c)
    assert rms(run_weight(c, lse, 900)[0], oracle_weight(c, lse, 900)[0]) < LIMIT8


def held(x, dtype, parts):
    """x as a sum of so many values of `dtype`, over the power of two that keeps a row's largest below 2^14."""
    up = 2.0 ** (13 - torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))))
    rest, out = x * up, torch.zeros_like(x)
    for _ in range(parts):
        part = rest.to(DTYPES[dtype]).double()
        out, rest = out + part, rest - part
    return out / up


@pytest.mark.parametrize("dtype,cache,scale_len,k_cache", CODES)
def test_the_bound_shows_a_part_that_is_left_out(dtype, cache, scale_len, k_cache):
    """On the CPU, with the queries that the kernel would hold in the oracle's place of the given ones: two parts are well below the
    bound, one is well above it."""
    c = case(dtype, cache, scale_len, k_cache)
    lse = row_lse(c)
    want = oracle_weight(c, lse, 900)[0]
    for parts in (1, 2):
        d = case(dtype, cache, scale_len, k_cache)
        if scale_len > 1:
            s = c.ckv_scale.double()
            d.q_nope = held(c.q_nope.double() / s, "f16", parts) * s
        else:
            s = c.ckv_scale.double() * (1.0 if c.k_scale is None else 1.0 / c.k_scale.double())
            d.q_rope = held(c.q_rope.double() * s, dtype if k_cache is None else "f16", parts) / s
        error = rms(oracle_weight(d, lse, 900)[0], want)
        assert (error > 3 * LIMIT8) if parts == 1 else (error < LIMIT8 / 3)
