"""Refusals of mla_key_weight at the ends of its ranges, without a GPU."""
import ctypes

import pytest

from attention_prologue_kv_gb300 import _native as N
from test_abi_cache_ops import lib, weight  # noqa: F401

# Addresses that stay apart: inputs below 2^44, the weights above.
FAR = dict(q_nope=1 << 40, q_rope=1 << 41, query_start=1 << 42, key_length=(1 << 42) + (1 << 20), block_table=(1 << 42) + (1 << 30),
           ckv_cache=1 << 43, k_cache=(1 << 43) + (1 << 38), lse=3 << 42, workspace=0)


def call(lib, T, H, Dv=8, Dk=8, **kw):  # noqa: F811
    step = dict(T=T, H=H, N=1, Dv=Dv, Dk=Dk, q_nope_token_stride=Dv * H, q_nope_head_stride=Dv, q_rope_token_stride=Dk * H,
                q_rope_head_stride=Dk, **FAR)
    return lib.mla_key_weight(ctypes.byref(weight(step, **dict(dict(weight=1 << 45, past=0), **kw))), None)


# 31 bits hold a key's place among the tokens, up to 255 behind the last one, and a query box's rows, up to 127 behind.
@pytest.mark.parametrize("T,H,want", [
    ((1 << 31) - 1, 1, N.KVR_ERR_SHAPE), ((1 << 31) - 511, 1, N.KVR_ERR_SHAPE), ((1 << 31) - 512, 1, N.KVR_ERR_NULL),
    ((1 << 24) - 1, 128, N.KVR_ERR_SHAPE), ((1 << 24) - 4, 128, N.KVR_ERR_NULL)])
def test_most_rows_on_the_tensor_cores(lib, T, H, want):  # noqa: F811
    assert call(lib, T, H) == want   # (KVR_ERR_NULL: as far as the workspace, which is looked at behind the limits)


# Without weights to add to, past_stride is not looked at: NULL is no address that `weight` and `past` share.
@pytest.mark.parametrize("kw", [dict(weight_len=0, weight_stride=8, past_stride=0), dict(weight_len=64, weight_stride=64, past_stride=0)])
def test_neither_weight_nor_past(lib, kw):  # noqa: F811
    a = weight(dict(workspace=0), **dict(dict(weight=0, past=0), **kw))
    assert lib.mla_key_weight(ctypes.byref(a), None) == N.KVR_ERR_NULL   # (the workspace; `weight` where it has room for keys)
