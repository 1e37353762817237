"""Seeded random configurations of mla_attention, kv_cache_read and query_rope against the oracle, within the bounds of
the targeted tests: lengths, heads, pages, modes, types, scales, widths, strides, masks and holes that no list pairs up.
And codes where a sequence's rows (token, head) fill both CTAs of a pair and several row tiles."""
import numpy as np
import pytest
import torch

import test_gpu_cache_read
import test_gpu_query_rope
from attention_helpers import check_mla, half_step, mla_case, on_tensor_cores, oracle_mla, rounded_query, run_mla

pytestmark = pytest.mark.gpu

CODES8 = ["int8", "fp8_e4m3fn", "fp8_e5m2"]


def check(c):
    """check_mla against the query as the kernel rounds it. Where the weights are halves, a weight below 2^-14 of the format
    is off by up to 2^-25, half of a half's last step, and the row's largest one is at least 2^7 there: 2^-32 of it a key, so
    K 2^-32 max |value| of the output, which is at most u * that / u where check_mla takes at least u A."""
    tc = on_tensor_cores(c)
    per_channel = any(s is not None and s.numel() > 1 for s in (c.ckv_scale, c.k_scale))
    out, lse, st, A, B = oracle_mla(c, *(rounded_query(c) if per_channel and tc else (None, None)))
    if tc and (c.ckv.element_size() == 1 or c.q_nope.dtype == torch.float16):
        used = np.nan_to_num(c.ckv.double().numpy(), nan=0.0, posinf=0.0, neginf=0.0)
        most = np.abs(used).max() if c.ckv_scale is None else np.abs(used / c.ckv_scale.double().numpy()).max()
        A = A + int(c.key_length.max()) * 2.0 ** -32 * most / half_step(c.q_nope.dtype)
    check_mla(c, run_mla(c), (out, lse, st, A, B), p_rounded=tc)


def log_int(r, lo, hi):
    return int(round(lo * (hi / lo) ** r.random()))


def mla_config(i):
    r = np.random.default_rng(7000 + i)
    dtype = str(r.choice(["bf16", "f16"]))
    cache = str(r.choice([dtype, dtype] + CODES8))
    k_cache = str(r.choice([dtype, dtype] + CODES8))
    Dv, Dk = [(512, 64), (512, 64), (512, 64), (256, 64), (448, 32), (64, 16), (136, 24), (20, 10)][int(r.integers(8))]
    H, n = log_int(r, 1, 130), int(r.integers(1, 9))
    new = [int(x) for x in r.integers(0, log_int(r, 2, 40), n)]
    keys = [int(r.integers(0, 1 + log_int(r, 1, 900))) for _ in range(n)]
    while sum(new) * H * max(keys) > 3_000_000:   # the oracle's time
        keys = [k // 2 for k in keys]
    mode = str(r.choice(["Norm", "PA_BSND", "PA_BSND", "PA_BLK_BSND"]))
    block = int(r.choice([1, 3, 8, 16, 24, 32, 64, 100, 128]))
    holes = [] if mode == "Norm" or r.random() < 0.5 else [(s, b) for s, k in enumerate(keys) for b in range(-(-k // block)) if r.random() < 0.2]
    scale_len, k_scale_len = (int(x) for x in r.integers(0, 2, 2))
    per_channel = (scale_len == 0 and cache in CODES8) or (k_scale_len == 0 and k_cache in CODES8)
    return dict(new=new, keys=keys, H=H, Dv=Dv, Dk=Dk, block_size=block, dtype=dtype, cache=cache, k_cache=k_cache, scale_len=scale_len,
                k_scale_len=k_scale_len, seed=7100 + i, causal=bool(r.random() < 0.7), mode=mode, gap=int(r.integers(0, 4)), holes=holes,
                spread=float(r.choice([0.3, 1.0, 4.0])), pad=int(r.choice([0, 0, 8] if per_channel else [0, 0, 8, 3])))


@pytest.mark.parametrize("i", range(80))
def test_mla_random_configurations(i):
    check(mla_case(**mla_config(i)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache,k_cache", [("int8", None), ("fp8_e4m3fn", "fp8_e4m3fn"), ("fp8_e5m2", "int8"), (None, "int8"), (None, "fp8_e4m3fn")])
@pytest.mark.parametrize("scale_len", [1, 0])
@pytest.mark.parametrize("new,keys,H", [([1], [130], 128), ([5, 1], [190, 65], 50), ([3, 40, 1], [64, 300, 1], 20)])
def test_codes_in_both_ctas_of_a_pair(new, keys, H, scale_len, cache, k_cache, dtype):
    """128, 250 and 800 rows of a sequence: rows 64 to 127 of a tile are the second CTA's, with their prepared queries."""
    check(mla_case(new, keys, H, dtype=dtype, cache=cache, k_cache=k_cache, scale_len=scale_len, k_scale_len=scale_len, seed=70))


@pytest.mark.parametrize("i", range(40))
def test_read_random_configurations(i):
    r = np.random.default_rng(8000 + i)
    dtype, mode = str(r.choice(["bf16", "f16"])), str(r.choice(["Norm", "PA_BSND", "PA_BLK_BSND"]))
    Dv, Dk = [(512, 64), (512, 64), (256, 32), (40, 8), (17, 3)][int(r.integers(5))]
    test_gpu_cache_read.check(int(r.integers(1, 9)), int(r.integers(1, 200)), mode, Dv, Dk, int(r.integers(1, 140)), dtype,
                              str(r.choice([dtype] + CODES8)), str(r.choice([dtype] + CODES8)), bool(r.random() < 0.5),
                              int(r.choice([0, 0, 8, 16, 3])), 8100 + i, bool(r.random() < 0.3))


@pytest.mark.parametrize("i", range(40))
def test_rope_random_configurations(i):
    r = np.random.default_rng(9000 + i)
    D = int(r.choice([2, 6, 16, 32, 64, 64, 72, 128, 256]))
    axes = int(r.integers(1, 6))
    cuts = sorted(int(x) for x in r.integers(0, D // 2 + 1, axes - 1))
    sections = [b - a for a, b in zip([0] + cuts, cuts + [D // 2])]
    test_gpu_query_rope.check(log_int(r, 1, 700), log_int(r, 1, 130), D, sections, str(r.choice(["bf16", "f16"])),
                              str(r.choice(["interleave", "half"])), float(r.choice([1e4, 5e5])), int(r.choice([0, 0, 8, 3, 64])),
                              bool(r.random() < 0.7), seed=9100 + i)
