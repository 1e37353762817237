"""Refusals of mla_attention at the ends of its ranges, without a GPU, and the arithmetic behind them."""
import ctypes
import random

import pytest

from attention_prologue_kv_gb300 import _native as N
from attention_prologue_kv_gb300.build import build
from test_abi_attention_step import mla_args


@pytest.fixture(scope="module")
def lib():
    build()
    return N.lib()


def narrow(T, H, **kw):
    """Rows of 8 + 8 channels, whose addresses and sizes stay apart: inputs below 2^40, out and workspace above."""
    a = dict(T=T, H=H, Dv=8, Dk=8, q_nope=1 << 40, q_nope_token_stride=8 * H, q_nope_head_stride=8, q_rope=1 << 42,
             q_rope_token_stride=8 * H, q_rope_head_stride=8, out=1 << 44, out_token_stride=8 * H, out_head_stride=8,
             ckv_cache=1 << 46, k_cache=1 << 47, block_table=1 << 48, query_start=1 << 49, key_length=1 << 50, workspace=1 << 52,
             workspace_bytes=1 << 40)
    a.update(kw)
    return mla_args(**a)


# (T, H, N, keys of a sequence) whose work does not fit 64 bits, and ones a step below
@pytest.mark.parametrize("T,H,n,keys,fits", [
    (32767, 65536, 1, 1 << 24, False),           # 2^24 row tiles x 2^16 heads x 2^24 keys = 2^64
    (32767, 65536, 1, 1 << 20, True),
    (1 << 20, 128, 1 << 12, 1 << 24, False),     # 2^20 x 2^7 x 2^12 x 2^24
    (1 << 20, 128, 1 << 10, 1 << 20, True),      # a million tokens, a thousand sequences with room for a million keys each
    (4096, 128, 4096, 1 << 24, True),            # a decode batch with room for the most keys
    ((1 << 31) - 1, 1, 1, 16, True)])
def test_work_beyond_64_bits_is_refused(lib, T, H, n, keys, fits):
    a = narrow(T, H, N=n, cache_d0=1 << 20, cache_d1=16, max_blocks=keys // 16)
    assert (lib.kvr_mla_attention_workspace(ctypes.byref(a)) > 0) == fits
    if not fits:
        assert lib.mla_attention(ctypes.byref(a), None) == N.KVR_ERR_SHAPE


@pytest.mark.parametrize("n,ok", [((1 << 31) - 513, True), ((1 << 31) - 512, False), ((1 << 31) - 1, False)])
def test_the_most_sequences(lib, n, ok):
    """The schedule rounds N up to its threads, 256 a half, in 32 bits."""
    assert (lib.kvr_mla_attention_workspace(ctypes.byref(narrow(4, 8, N=n, cache_d0=8, cache_d1=16, max_blocks=1))) > 0) == ok


def share(total, which, active):
    """Where share `which` begins, in the kernel's steps."""
    each = total // active
    low = (total - each * active) * which
    assert each * which < 1 << 63 and low < 1 << 32
    return each * which + low // active


def test_shares_are_those_of_the_product():
    """total * which // active, also where the product passes 64 bits."""
    r = random.Random(1)
    for _ in range(20000):
        active = r.randint(1, 256)
        total = r.randint(0, 1 << r.randint(1, 62))
        which = r.randint(0, active - 1)
        assert share(total, which, active) == total * which // active
