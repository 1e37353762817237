"""The C ABI of drafted trees and bounded caches without a GPU: structure layouts against a C compiler, and the refusals that
the host makes before any CUDA call (pointers are never dereferenced)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from attention_prologue_kv_gb300 import _native as N
from attention_prologue_kv_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
M = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build()
    return N.lib()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_struct_layout_matches_c(tmp_path):
    types = (("kvr_tree_args", N.TreeArgs), ("kvr_mla_tree_args", N.MlaTreeArgs), ("kvr_key_weight_args", N.KeyWeightArgs),
             ("kvr_select_args", N.SelectArgs), ("kvr_compact_args", N.CompactArgs))
    body = "".join('printf("%s %%zu\\n", sizeof(%s));' % (t, t) for t, _ in types)
    body += "".join('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (t, f[0], t, f[0]) for t, c in types for f in c._fields_)
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvr.h"\nint main(void) {%s return 0;}' % body)
    exe = tmp_path / "probe"
    inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-I", inc, str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for t, c in types:
        assert int(got[t]) == ctypes.sizeof(c)
        for f in c._fields_:
            assert int(got["%s.%s" % (t, f[0])]) == getattr(c, f[0]).offset, (t, f[0])


def tree(**kw):
    a = dict(T=10, N=2, query_start=M, parent=2 * M, position_start=3 * M, tree_mask=4 * M, mask_words=1, positions=5 * M)
    a.update(kw)
    return N.TreeArgs(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), N.KVR_ERR_SHAPE), (dict(N=-1), N.KVR_ERR_SHAPE), (dict(mask_words=0), N.KVR_ERR_SHAPE),
    (dict(mask_words=65), N.KVR_ERR_SHAPE), (dict(T=1 << 60, mask_words=8), N.KVR_ERR_SHAPE),
    (dict(query_start=0), N.KVR_ERR_NULL), (dict(parent=0), N.KVR_ERR_NULL), (dict(tree_mask=0), N.KVR_ERR_NULL),
    (dict(position_start=0), N.KVR_ERR_NULL), (dict(parent=2 * M + 4), N.KVR_ERR_SHAPE),
    (dict(tree_mask=4 * M + 4), N.KVR_ERR_SHAPE), (dict(dev_status=6 * M + 2), N.KVR_ERR_SHAPE),
    (dict(tree_mask=2 * M + 72), N.KVR_ERR_ALIAS), (dict(positions=4 * M + 8), N.KVR_ERR_ALIAS),
    (dict(dev_status=5 * M), N.KVR_ERR_ALIAS), (dict(T=0, parent=0), N.KVR_OK), (dict(N=0), N.KVR_OK)])
def test_draft_tree_refusals(lib, kw, want):
    assert lib.draft_tree(ctypes.byref(tree(**kw)), None) == want


def step(**kw):
    a = dict(q_nope=M, q_rope=2 * M, dtype=0, T=4, H=2, Dv=512, Dk=64, q_nope_token_stride=1024, q_nope_head_stride=512,
             q_rope_token_stride=128, q_rope_head_stride=64, N=2, query_start=3 * M, key_length=4 * M, mode=1, cache_d0=8,
             cache_d1=16, block_table=5 * M, max_blocks=4, ckv_cache=6 * M, ckv_dtype=0, k_cache=8 * M, k_dtype=0,
             softmax_scale=0.1, causal=1, out=9 * M, out_token_stride=1024, out_head_stride=512, lse=10 * M, workspace=12 * M,
             workspace_bytes=0)
    a.update(kw)
    return N.MlaArgs(**a)


@pytest.mark.parametrize("kw,words,mask,want", [
    (dict(), 0, 11 * M, N.KVR_ERR_SHAPE), (dict(), -1, 11 * M, N.KVR_ERR_SHAPE), (dict(), 1, 0, N.KVR_ERR_NULL),
    (dict(), 1, 11 * M + 4, N.KVR_ERR_SHAPE), (dict(), 1 << 58, 11 * M, N.KVR_ERR_SHAPE), (dict(), 1, 9 * M + 8, N.KVR_ERR_ALIAS),
    (dict(), 1, 10 * M, N.KVR_ERR_ALIAS), (dict(T=-1), 1, 11 * M, N.KVR_ERR_SHAPE), (dict(mode=7), 1, 11 * M, N.KVR_ERR_MODE),
    (dict(out=0), 1, 11 * M, N.KVR_ERR_NULL), (dict(workspace=0), 1, 11 * M, N.KVR_ERR_NULL), (dict(T=0), 1, 0, N.KVR_OK)])
def test_tree_attention_refusals(lib, kw, words, mask, want):
    a = N.MlaTreeArgs(attention=step(**kw), tree_mask=mask, mask_words=words)
    assert lib.mla_tree_attention(ctypes.byref(a), None) == want


def weight(step_kw=None, **kw):
    a = dict(step=step(**dict(dict(out=0), **(step_kw or {}))), weight=11 * M, weight_stride=64, weight_len=64, past=13 * M,
             past_stride=64, decay=1.0)
    a.update(kw)
    return N.KeyWeightArgs(**a)


@pytest.mark.parametrize("step_kw,kw,want", [
    (None, dict(weight_len=-1), N.KVR_ERR_SHAPE), (None, dict(weight_stride=63), N.KVR_ERR_SHAPE),
    (None, dict(past_stride=63), N.KVR_ERR_SHAPE), (None, dict(decay=float("nan")), N.KVR_ERR_SHAPE),
    (None, dict(weight=11 * M + 2), N.KVR_ERR_SHAPE), (None, dict(weight=0), N.KVR_ERR_NULL),
    (None, dict(weight_stride=1 << 61), N.KVR_ERR_SHAPE),
    (dict(lse=0), dict(), N.KVR_ERR_NULL), (dict(q_rope=0), dict(), N.KVR_ERR_NULL), (dict(key_length=0), dict(), N.KVR_ERR_NULL),
    (None, dict(weight=10 * M), N.KVR_ERR_ALIAS), (None, dict(past=11 * M + 4), N.KVR_ERR_ALIAS),
    (None, dict(past=11 * M, past_stride=65), N.KVR_ERR_ALIAS), (None, dict(weight=6 * M + 16), N.KVR_ERR_ALIAS),
    (dict(dev_status=11 * M), dict(), N.KVR_ERR_ALIAS), (dict(dtype=2), dict(), N.KVR_ERR_DTYPE),
    (dict(Dv=0), dict(), N.KVR_ERR_SHAPE), (dict(ckv_dtype=2), dict(), N.KVR_ERR_NULL), (dict(H=0), dict(), N.KVR_OK),
    (dict(T=0), dict(), N.KVR_OK)])
def test_key_weight_refusals(lib, step_kw, kw, want):
    assert lib.mla_key_weight(ctypes.byref(weight(step_kw, **kw)), None) == want


def test_key_weight_refuses_work_that_64_bits_cannot_count(lib):
    kw = dict(T=1 << 30, H=1, q_nope_token_stride=512, q_rope_token_stride=64, q_nope_head_stride=512, q_rope_head_stride=64, mode=1,
              cache_d0=1, cache_d1=1 << 24, max_blocks=1, q_nope=0, workspace=0)
    far = dict(q_nope=1 << 50, q_rope=1 << 51, query_start=1 << 52, key_length=3 << 51, block_table=1 << 53, ckv_cache=3 << 52,
               k_cache=1 << 54, lse=3 << 53)
    out = dict(weight=1 << 55, weight_len=1 << 24, weight_stride=1 << 24, past=0)
    # (2^30 / 32 + 1) * (2^16 + 1) * N against 2^62: N = 2^21 is too many, 2^21 - 2^16 would be launched, had it a workspace
    for n, want in ((1 << 21, N.KVR_ERR_SHAPE), ((1 << 21) - (1 << 16), N.KVR_ERR_NULL)):
        assert lib.mla_key_weight(ctypes.byref(weight(dict(kw, N=n, **far), **out)), None) == want


def select(**kw):
    a = dict(weight=M, weight_stride=100, weight_len=100, N=3, key_length=2 * M, keep=20, sink=2, recent=5, kept=3 * M,
             kept_length=4 * M, kept_weight=5 * M, kept_weight_stride=20, kept_weight_len=20)
    a.update(kw)
    return N.SelectArgs(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), N.KVR_ERR_SHAPE), (dict(N=1 << 27), N.KVR_ERR_SHAPE), (dict(weight_len=-1), N.KVR_ERR_SHAPE),
    (dict(weight_stride=99), N.KVR_ERR_SHAPE), (dict(weight_len=1 << 31, weight_stride=1 << 31), N.KVR_ERR_SHAPE),
    (dict(keep=0), N.KVR_ERR_SHAPE), (dict(keep=1 << 31), N.KVR_ERR_SHAPE), (dict(sink=-1), N.KVR_ERR_SHAPE),
    (dict(recent=-1), N.KVR_ERR_SHAPE), (dict(sink=16), N.KVR_ERR_SHAPE), (dict(recent=19), N.KVR_ERR_SHAPE),
    (dict(sink=1 << 62, recent=1 << 62), N.KVR_ERR_SHAPE), (dict(kept_weight_len=19), N.KVR_ERR_SHAPE),
    (dict(kept_weight_stride=19), N.KVR_ERR_SHAPE), (dict(weight=0), N.KVR_ERR_NULL), (dict(key_length=0), N.KVR_ERR_NULL),
    (dict(kept=0), N.KVR_ERR_NULL), (dict(kept_length=0), N.KVR_ERR_NULL), (dict(kept=3 * M + 4), N.KVR_ERR_SHAPE),
    (dict(weight=M + 2), N.KVR_ERR_SHAPE), (dict(kept=M + 8), N.KVR_ERR_ALIAS), (dict(kept_weight=M + 1196), N.KVR_ERR_ALIAS),
    (dict(kept_length=3 * M + 472), N.KVR_ERR_ALIAS), (dict(dev_status=2 * M), N.KVR_ERR_ALIAS), (dict(N=0, weight=0), N.KVR_OK)])
def test_select_refusals(lib, kw, want):
    assert lib.kv_cache_select(ctypes.byref(select(**kw)), None) == want


# A key's number and the end of its CTA's share, both rounded up, are counted in 31 bits.
def test_select_longest(lib):
    far = dict(weight=1 << 50, key_length=1 << 51, kept=1 << 52, kept_weight=0, N=1)
    for length in ((1 << 30) + 1, (1 << 31) - 1):
        a = select(weight_len=length, weight_stride=length, kept_length=1 << 53, **far)
        assert lib.kv_cache_select(ctypes.byref(a), None) == N.KVR_ERR_SHAPE
    # (as far as a null pointer, which is looked at behind the limits)
    assert lib.kv_cache_select(ctypes.byref(select(weight_len=1 << 30, weight_stride=1 << 30, kept_length=0, **far)), None) == N.KVR_ERR_NULL


def compact(**kw):
    a = dict(ckv_cache=M, ckv_dtype=0, k_cache=3 * M, k_dtype=0, mode=1, cache_d0=8, cache_d1=16, block_table=4 * M, max_blocks=4,
             N=2, Dv=512, Dk=64, kept=5 * M, kept_len=7, kept_length=6 * M, start=7 * M)
    a.update(kw)
    return N.CompactArgs(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(mode=3), N.KVR_ERR_MODE), (dict(ckv_dtype=9), N.KVR_ERR_DTYPE), (dict(k_dtype=-1), N.KVR_ERR_DTYPE),
    (dict(N=-1), N.KVR_ERR_SHAPE), (dict(Dv=0), N.KVR_ERR_SHAPE), (dict(Dk=-1), N.KVR_ERR_SHAPE), (dict(kept_len=-1), N.KVR_ERR_SHAPE),
    (dict(cache_d1=0), N.KVR_ERR_SHAPE), (dict(mode=0, N=9), N.KVR_ERR_SHAPE), (dict(ckv_cache=0), N.KVR_ERR_NULL),
    (dict(k_cache=0), N.KVR_ERR_NULL), (dict(kept=0), N.KVR_ERR_NULL), (dict(kept_length=0), N.KVR_ERR_NULL),
    (dict(block_table=0), N.KVR_ERR_NULL), (dict(ckv_cache=M + 1), N.KVR_ERR_SHAPE), (dict(kept=5 * M + 4), N.KVR_ERR_SHAPE),
    (dict(kept=M + 8), N.KVR_ERR_ALIAS), (dict(k_cache=M + 1024), N.KVR_ERR_ALIAS), (dict(start=M), N.KVR_ERR_ALIAS),
    (dict(dev_status=3 * M), N.KVR_ERR_ALIAS), (dict(N=0), N.KVR_OK), (dict(kept_len=0), N.KVR_OK)])
def test_compact_refusals(lib, kw, want):
    assert lib.kv_cache_compact(ctypes.byref(compact(**kw)), None) == want


def test_null_arguments(lib):
    for f in (lib.draft_tree, lib.mla_tree_attention, lib.mla_key_weight, lib.kv_cache_select, lib.kv_cache_compact):
        assert f(None, None) == N.KVR_ERR_NULL
    assert lib.kvr_mla_key_weight_workspace(None) == 0


def test_python_refuses_host_tensors():
    import attention_prologue_kv_gb300 as kvr
    i, f = torch.zeros(2, dtype=torch.int64), torch.zeros(2, 4)
    b = torch.zeros(1, 2, 1, 512, dtype=torch.bfloat16)
    for call in (lambda: kvr.draft_tree(i, i, i.view(2, 1)), lambda: kvr.kv_cache_select(f, i, i.view(2, 1), i),
                 lambda: kvr.kv_cache_compact(b, b, i.view(2, 1), i.view(2, 1), i),
                 lambda: kvr.mla_key_weight(b[0], b[0], b, b, i.view(1, 2), i, i[:1], f, f, softmax_scale=1.0)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
