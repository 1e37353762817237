"""GPU parity of mla_attention against the float64 oracle, within the bounds that check_mla derives."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
from attention_prologue_kv_gb300 import _native as N
from attention_helpers import SENTINEL, check_mla, half_step, mla_case, on_tensor_cores, oracle_mla, rounded_query, run_mla

pytestmark = pytest.mark.gpu


def check(c):
    per_channel = any(s is not None and s.numel() > 1 for s in (c.ckv_scale, c.k_scale))
    got = run_mla(c)
    tc = on_tensor_cores(c)
    q = rounded_query(c) if per_channel and tc else [None, None]
    check_mla(c, got, oracle_mla(c, *q), p_rounded=tc)
    if per_channel:   # and near the definition itself
        want = oracle_mla(c)[0]
        fin = want != SENTINEL
        assert np.linalg.norm((got[0] - want)[fin]) <= 4 * torch.finfo(c.q_nope.dtype).eps * np.linalg.norm(want[fin])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,keys,H", [
    ([1], [1], 1), ([1], [64], 16), ([1], [65], 128), ([1], [1000], 16), ([1, 1, 1], [1, 63, 129], 40), ([5], [5], 3),
    ([130], [130], 1), ([7, 1, 0, 3], [300, 9, 20, 3], 20), ([33], [200], 7), ([2, 2], [700, 64], 130), ([1] * 40, list(range(1, 41)), 2)])
def test_lengths_and_heads(new, keys, H, dtype):
    check(mla_case(new, keys, H, dtype=dtype, seed=H))


@pytest.mark.parametrize("block_size", [1, 3, 16, 32, 64, 100, 128, 500])
def test_block_sizes(block_size):
    check(mla_case([3, 1], [401, 130], 8, block_size=block_size, seed=block_size))


@pytest.mark.parametrize("mode", ["Norm", "PA_BLK_BSND"])
def test_modes(mode):
    check(mla_case([3, 1, 2], [401, 130, 64], 8, mode=mode, seed=1))


@pytest.mark.parametrize("causal", [True, False])
def test_masks(causal):
    """More new tokens than keys, no keys at all, rows behind the last sequence."""
    c = mla_case([9, 4, 1, 1], [5, 0, 0, 70], 6, causal=causal, gap=3, seed=2)
    out, lse, _ = check(c)
    assert (out[-3:] == SENTINEL).all() and (lse[-3:] == SENTINEL).all()
    if causal:
        assert (out[:4] == 0).all() and np.isneginf(lse[:4]).all()


def test_holes_in_the_block_table():
    check(mla_case([1, 4, 1], [200, 90, 33], 16, holes=[(0, 0), (0, 7), (1, 2), (1, 5), (2, 0), (2, 1), (2, 2)], seed=3))


def test_bad_metadata_leaves_sequences_out():
    c = mla_case([2, 1, 3, 1], [40, 50, 60, 33], 4, gap=4, seed=4)
    c.key_length[1] = -1
    c.key_length[2] = 10 ** 7
    check(c)
    c = mla_case([2, 1, 3, 1], [40, 50, 60, 33], 4, gap=4, seed=4)
    c.table[3, 1] = 10 ** 9
    c.table[0, 0] = -5
    check(c)
    c.query_start[4] = 10 ** 6
    check(c)
    c.query_start[:] = torch.tensor([2, 1, 3, 8, 8])
    check(c)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache", ["int8", "fp8_e4m3fn", "fp8_e5m2"])
@pytest.mark.parametrize("k8,scale_len", [(False, 1), (True, 1), (False, 0), (True, 0)])
def test_8_bit_caches(cache, dtype, k8, scale_len):
    check(mla_case([1, 5, 1], [190, 77, 64], 12, dtype=dtype, cache=cache, k_cache=cache if k8 else None, scale_len=scale_len,
                   k_scale_len=scale_len, seed=6))


@pytest.mark.parametrize("Dv,Dk", [(256, 32), (64, 8), (320, 64), (512, 16), (10, 6), (1, 1), (1000, 130), (504, 56)])
@pytest.mark.parametrize("cache", [None, "int8"])
def test_widths(Dv, Dk, cache):
    check(mla_case([3, 1], [150, 70], 5, Dv, Dk, cache=cache, seed=Dv))


@pytest.mark.parametrize("pad", [0, 8, 3])
def test_strided_queries(pad):
    check(mla_case([3, 1], [150, 70], 5, pad=pad, seed=pad))


@pytest.mark.parametrize("spread", [0.01, 30.0])
def test_flat_and_sharp_softmax(spread):
    check(mla_case([2], [700], 16, spread=spread, seed=8))


def test_long_context_of_one_token():
    check(mla_case([1], [20000], 8, block_size=128, seed=9))


def test_repeats_are_equal():
    """One GPU, the same inputs: the same bits."""
    c = mla_case([40, 1], [2000, 900], 24, block_size=64, seed=10)
    a, b = run_mla(c), run_mla(c)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_empty_problems():
    for T, H, n in ((0, 4, 2), (3, 0, 1), (3, 4, 0)):
        z = lambda *s: torch.full(s, SENTINEL, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        out = z(T, H, 512)
        kvr.mla_attention(z(T, H, 512), z(T, H, 64), z(2, 4, 1, 512), z(2, 4, 1, 64), torch.zeros(n, 2, device="cuda", dtype=torch.int64),
                          torch.zeros(n + 1, device="cuda", dtype=torch.int64), torch.zeros(n, device="cuda", dtype=torch.int64), out,
                          softmax_scale=1.0)
        torch.cuda.synchronize()
        assert (out == SENTINEL).all()


def test_most_keys():
    """2^24 keys (a table that names one block over and over: the softmax is that of the block alone) and one more.

    A part sums 2^24 / 76 keys, 16 an instruction into the output's sum and two at a time into a thread's share of l: fewer than 2^15
    additions of 2^-23 each, in the sum and in what it is divided by, so 2^-7 of the weights' sum of magnitudes."""
    d1, reps = 4096, 4096
    c = mla_case([1], [d1], H=3, block_size=d1, seed=31, causal=False)
    want, lse, _, A, B = oracle_mla(c)
    c.table = c.table[:, :1].repeat(1, reps + 1)
    c.key_length = torch.tensor([d1 * reps])
    out, ls, st = run_mla(c)
    assert st == 0
    u, ds = half_step(c.q_nope.dtype), 2.0 ** -17 * B + 2.0 ** -19   # (a score's error, as in check_mla)
    assert np.all(np.abs(out - want) <= (2 * ds[..., None] + 2.0 ** -7 + u) * A * (1 + u) + u * np.abs(want))
    assert np.all(np.abs(ls - lse - np.log(reps)) <= ds + 2.0 ** -8 + 2.0 ** -23 * np.abs(ls))
    c.key_length = torch.tensor([d1 * reps + 1])
    out, ls, st = run_mla(c)
    assert st == N.KVR_DEVERR_KEY_LENGTH and np.all(out == SENTINEL) and np.all(ls == SENTINEL)


@pytest.mark.parametrize("cache", ["int8", "fp8_e4m3fn"])
@pytest.mark.parametrize("block_size", [1, 3, 8, 24, 100])
def test_block_sizes_of_codes(block_size, cache):
    check(mla_case([3, 1], [401, 130], 8, block_size=block_size, cache=cache, k_cache=cache, seed=block_size))


@pytest.mark.parametrize("block_size", [3, 16, 64])
@pytest.mark.parametrize("k_cache,scale_len", [("int8", 1), ("fp8_e5m2", 0)])
def test_codes_in_the_rotary_part_alone(k_cache, scale_len, block_size):
    check(mla_case([3, 1], [401, 130], 8, block_size=block_size, k_cache=k_cache, k_scale_len=scale_len, seed=block_size))


@pytest.mark.parametrize("cache", [None, "int8"])
def test_many_sequences(cache):
    """More than a warp holds, most of them short, some without new tokens or keys."""
    new, keys = [(n * 7) % 4 for n in range(700)], [(n * 37) % 90 for n in range(700)]
    check(mla_case(new, keys, 3, cache=cache, seed=12))


@pytest.mark.parametrize("H", [65536, 65537])
def test_most_heads(H):
    check(mla_case([2], [70], H, Dv=8, Dk=8, seed=13))


def far(t, rows):
    """The cache `t` [d0, d1, 1, D] as the last blocks of one of `rows` rows that holds nothing else."""
    d0, d1, _, D = t.shape
    big = torch.empty(-(-rows // d1), d1, 1, D, dtype=t.dtype, device="cuda")
    big[-d0:].copy_(t)
    return big


@pytest.mark.parametrize("Dv,Dk,rows,cache", [
    (512, 64, 9 << 20, None), (512, 64, 9 << 20, "int8"), (8, 8, (1 << 31) + 1000, None), (16, 16, (1 << 31) + 1000, "int8")])
def test_far_rows(Dv, Dk, rows, cache):
    """Offsets behind 2^32 elements, row numbers behind 2^31: the same bits as near the cache's begin."""
    c = mla_case([3, 1], [401, 130], 8, Dv, Dk, block_size=32, cache=cache, k_cache=cache, seed=14)
    if torch.cuda.mem_get_info()[0] < 2 * rows * (Dv + Dk) * c.ckv.element_size():
        pytest.skip("not enough memory on this GPU")
    want = run_mla(c)
    d0 = c.ckv.shape[0]
    c.ckv, c.k = far(c.ckv, rows), far(c.k, rows)
    c.table = torch.where(c.table < 0, c.table, c.table + (c.ckv.shape[0] - d0))
    got = run_mla(c)
    assert got[2] == 0
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    index = torch.tensor([rows - 1, rows - 33, -1])
    out = torch.full((3, Dv + Dk), SENTINEL, device="cuda", dtype=c.q_nope.dtype)
    kvr.kv_cache_read(c.ckv, c.k, index.cuda(), out, ckv_scale=None if c.ckv_scale is None else c.ckv_scale.cuda(),
                      k_scale=None if c.k_scale is None else c.k_scale.cuda())
    near = torch.full_like(out, SENTINEL)
    kvr.kv_cache_read(c.ckv[-d0:], c.k[-d0:], (index - (c.ckv.shape[0] - d0) * 32).clamp(min=-1).cuda(), near,
                      ckv_scale=None if c.ckv_scale is None else c.ckv_scale.cuda(),
                      k_scale=None if c.k_scale is None else c.k_scale.cuda())
    assert torch.equal(out.view(torch.int16), near.view(torch.int16))
    c.ckv = c.k = None
    torch.cuda.empty_cache()   # tens of GB
