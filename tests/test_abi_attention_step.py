"""The C ABI of query_rope, kv_cache_read and mla_attention without a GPU:
structure layouts against a C compiler, and the refusals that the host makes
before any CUDA call (pointers are never dereferenced)."""
import ctypes
import os
import shutil
import subprocess

import pytest

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
    types = (("kvr_rope_args", N.RopeArgs), ("kvr_read_args", N.ReadArgs), ("kvr_mla_args", N.MlaArgs))
    body = "".join('printf("%s %%zu\\n", sizeof(%s));' % (t, t) for t, _ in types)
    body += "".join('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (t, f[0], t, f[0]) for t, c in types for f in c._fields_)
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvr.h"\nint main(void) {%s printf("axes %%d\\n", KVR_MAX_AXES);'
                   'printf("query %%d\\n", KVR_DEVERR_QUERY); return 0;}' % body)
    exe = tmp_path / "probe"
    inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-I", inc, str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for t, c in types:
        assert int(got[t]) == ctypes.sizeof(c)
        for f in c._fields_:
            assert int(got["%s.%s" % (t, f[0])]) == getattr(c, f[0]).offset, (t, f[0])
    assert int(got["axes"]) == N.KVR_MAX_AXES and int(got["query"]) == N.KVR_DEVERR_QUERY


def rope_args(**kw):
    sections = kw.pop("sections", (16, 16))
    arr = (ctypes.c_int64 * 9)(*sections) if sections is not None else None
    a = dict(q=M, dtype=N.KVR_BF16, T=3, H=2, D=64, q_token_stride=128, q_head_stride=64, positions=2 * M, axes=2, sections=arr,
             base=10000.0, half_pairs=0, out=3 * M, out_token_stride=128, out_head_stride=64, cos_out=None, sin_out=None)
    a.update(kw)
    r = N.RopeArgs(**a)
    r._keep = arr
    return r


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=N.KVR_INT8), N.KVR_ERR_DTYPE), (dict(D=63), N.KVR_ERR_SHAPE), (dict(D=0), N.KVR_ERR_SHAPE),
    (dict(D=258), N.KVR_ERR_SHAPE), (dict(T=-1), N.KVR_ERR_SHAPE), (dict(H=-1), N.KVR_ERR_SHAPE), (dict(axes=0), N.KVR_ERR_SHAPE),
    (dict(axes=9), N.KVR_ERR_SHAPE), (dict(sections=(16, 15)), N.KVR_ERR_SHAPE), (dict(sections=(33, -1)), N.KVR_ERR_SHAPE),
    (dict(sections=None), N.KVR_ERR_NULL), (dict(base=0.99), N.KVR_ERR_SHAPE), (dict(base=float("inf")), N.KVR_ERR_SHAPE),
    (dict(base=float("nan")), N.KVR_ERR_SHAPE), (dict(q=None), N.KVR_ERR_NULL), (dict(out=None), N.KVR_ERR_NULL),
    (dict(positions=None), N.KVR_ERR_NULL), (dict(cos_out=4 * M), N.KVR_ERR_NULL), (dict(positions=2 * M + 4), N.KVR_ERR_SHAPE),
    (dict(q=M + 1), N.KVR_ERR_SHAPE), (dict(q_token_stride=-1), N.KVR_ERR_SHAPE), (dict(out=M + 64), N.KVR_ERR_ALIAS),
    (dict(out=2 * M), N.KVR_ERR_ALIAS), (dict(out_head_stride=32), N.KVR_ERR_ALIAS), (dict(out_token_stride=64), N.KVR_ERR_ALIAS),
    (dict(cos_out=4 * M, sin_out=4 * M + 64), N.KVR_ERR_ALIAS), (dict(T=1 << 40, H=1 << 10), N.KVR_ERR_SHAPE),
    (dict(T=0, q=None, out=None, positions=None), N.KVR_OK), (dict(H=0, q=None, out=None), N.KVR_OK)])
def test_rope_refusals(lib, kw, want):
    assert lib.query_rope(ctypes.byref(rope_args(**kw)), None) == want


def read_args(**kw):
    a = dict(ckv_cache=M, ckv_dtype=N.KVR_BF16, ckv_scale=None, ckv_scale_len=0, k_cache=8 * M, k_dtype=N.KVR_BF16, k_scale=None,
             k_scale_len=0, mode=1, cache_d0=8, cache_d1=16, index=16 * M, B=2, S=3, Dv=512, Dk=64, out=32 * M,
             out_dtype=N.KVR_BF16, out_row_stride=0, dev_status=None)
    a.update(kw)
    return N.ReadArgs(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(mode=3), N.KVR_ERR_MODE), (dict(out_dtype=N.KVR_INT8), N.KVR_ERR_DTYPE), (dict(ckv_dtype=N.KVR_F16), N.KVR_ERR_DTYPE),
    (dict(k_dtype=7), N.KVR_ERR_DTYPE), (dict(B=-1), N.KVR_ERR_SHAPE), (dict(S=-1), N.KVR_ERR_SHAPE), (dict(Dv=0), N.KVR_ERR_SHAPE),
    (dict(Dk=-1), N.KVR_ERR_SHAPE), (dict(cache_d0=0), N.KVR_ERR_SHAPE), (dict(out_row_stride=575), N.KVR_ERR_SHAPE),
    (dict(mode=0, cache_d0=1), N.KVR_ERR_SHAPE), (dict(ckv_dtype=N.KVR_INT8), N.KVR_ERR_NULL),
    (dict(ckv_scale=64 * M, ckv_scale_len=1), N.KVR_ERR_NULL), (dict(k_dtype=N.KVR_FP8_E5M2), N.KVR_ERR_NULL),
    (dict(ckv_dtype=N.KVR_INT8, ckv_scale=64 * M, ckv_scale_len=3), N.KVR_ERR_SHAPE),
    (dict(ckv_dtype=N.KVR_INT8, ckv_scale=64 * M + 2, ckv_scale_len=1), N.KVR_ERR_SHAPE),
    (dict(out=None), N.KVR_ERR_NULL), (dict(index=None), N.KVR_ERR_NULL), (dict(ckv_cache=None), N.KVR_ERR_NULL),
    (dict(k_cache=None), N.KVR_ERR_NULL), (dict(index=16 * M + 4), N.KVR_ERR_SHAPE), (dict(out=M + 2048), N.KVR_ERR_ALIAS),
    (dict(out=16 * M), N.KVR_ERR_ALIAS), (dict(cache_d0=1 << 40, cache_d1=1 << 20), N.KVR_ERR_SHAPE),
    (dict(B=0, out=None), N.KVR_OK), (dict(S=0, index=None), N.KVR_OK)])
def test_read_refusals(lib, kw, want):
    assert lib.kv_cache_read(ctypes.byref(read_args(**kw)), None) == want


def mla_args(**kw):
    a = dict(q_nope=M, q_rope=2 * M, dtype=N.KVR_BF16, T=4, H=8, Dv=512, Dk=64, q_nope_token_stride=4096, q_nope_head_stride=512,
             q_rope_token_stride=512, q_rope_head_stride=64, N=2, query_start=3 * M, key_length=4 * M, mode=1, cache_d0=8, cache_d1=16,
             block_table=5 * M, max_blocks=4, ckv_cache=6 * M, ckv_dtype=N.KVR_BF16, ckv_scale=None, ckv_scale_len=0, k_cache=8 * M,
             k_dtype=N.KVR_BF16, k_scale=None, k_scale_len=0, softmax_scale=0.1, causal=1, out=16 * M, out_token_stride=4096,
             out_head_stride=512, lse=None, workspace=64 * M, workspace_bytes=0, dev_status=None)
    a.update(kw)
    return N.MlaArgs(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(mode=9), N.KVR_ERR_MODE), (dict(dtype=N.KVR_FP8_E4M3FN), N.KVR_ERR_DTYPE), (dict(ckv_dtype=N.KVR_F16), N.KVR_ERR_DTYPE),
    (dict(T=-1), N.KVR_ERR_SHAPE), (dict(H=-2), N.KVR_ERR_SHAPE), (dict(N=-1), N.KVR_ERR_SHAPE), (dict(Dv=0), N.KVR_ERR_SHAPE),
    (dict(Dv=1025), N.KVR_ERR_SHAPE), (dict(Dk=0), N.KVR_ERR_SHAPE), (dict(Dk=257), N.KVR_ERR_SHAPE), (dict(max_blocks=-1), N.KVR_ERR_SHAPE),
    (dict(T=1 << 20, H=1 << 12), N.KVR_ERR_SHAPE), (dict(mode=0, cache_d0=1), N.KVR_ERR_SHAPE), (dict(softmax_scale=float("nan")), N.KVR_ERR_SHAPE),
    (dict(q_nope=None), N.KVR_ERR_NULL), (dict(q_rope=None), N.KVR_ERR_NULL), (dict(out=None), N.KVR_ERR_NULL),
    (dict(query_start=None), N.KVR_ERR_NULL), (dict(key_length=None), N.KVR_ERR_NULL), (dict(block_table=None), N.KVR_ERR_NULL),
    (dict(ckv_cache=None), N.KVR_ERR_NULL), (dict(k_cache=None), N.KVR_ERR_NULL), (dict(ckv_dtype=N.KVR_INT8), N.KVR_ERR_NULL),
    (dict(k_scale=32 * M, k_scale_len=1), N.KVR_ERR_NULL), (dict(key_length=4 * M + 4), N.KVR_ERR_SHAPE), (dict(lse=40 * M + 2), N.KVR_ERR_SHAPE),
    (dict(q_nope_head_stride=-8), N.KVR_ERR_SHAPE), (dict(out_head_stride=256), N.KVR_ERR_ALIAS), (dict(out=M), N.KVR_ERR_ALIAS),
    (dict(out=6 * M), N.KVR_ERR_ALIAS), (dict(lse=16 * M), N.KVR_ERR_ALIAS), (dict(workspace=16 * M, workspace_bytes=4096), N.KVR_ERR_ALIAS),
    (dict(workspace=None), N.KVR_ERR_NULL), (dict(), N.KVR_ERR_SHAPE),   # no room in the workspace
    (dict(workspace=64 * M + 8, workspace_bytes=1 << 40), N.KVR_ERR_SHAPE),
    (dict(workspace=64 * M + 16, workspace_bytes=1 << 24), N.KVR_ERR_SHAPE),   # its rows are written 32 bytes at a time
    (dict(cache_d0=1 << 40, cache_d1=1 << 20), N.KVR_ERR_SHAPE),
    (dict(T=0, q_nope=None), N.KVR_OK), (dict(H=0, q_nope=None), N.KVR_OK), (dict(N=0, query_start=None), N.KVR_OK)])
def test_mla_refusals(lib, kw, want):
    assert lib.mla_attention(ctypes.byref(mla_args(**kw)), None) == want


def test_null_arguments(lib):
    assert lib.query_rope(None, None) == lib.kv_cache_read(None, None) == lib.mla_attention(None, None) == N.KVR_ERR_NULL
    assert lib.kvr_mla_attention_workspace(None) == 0


def test_workspace_follows_the_arguments(lib):
    """Codes with a scale per channel need room for their prepared queries; rows that the plain kernel takes need none."""
    need = lambda **kw: lib.kvr_mla_attention_workspace(ctypes.byref(mla_args(**kw)))  # noqa: E731
    plain = need()
    assert plain > 0 and need(q_nope_head_stride=516, q_nope_token_stride=4200) == 0 and need(Dv=500) == 0 and need(T=-1) == 0
    codes = need(ckv_dtype=N.KVR_INT8, ckv_scale=32 * M, ckv_scale_len=512)
    assert codes >= plain + 4 * 8 * (512 * 2 + 4)
    # halves and one scale need no preparation
    half = dict(dtype=N.KVR_F16, k_dtype=N.KVR_F16, ckv_dtype=N.KVR_INT8, ckv_scale=32 * M, ckv_scale_len=1)
    assert need(**half) == plain


def test_binding_refuses_cpu_tensors():
    import torch
    import attention_prologue_kv_gb300 as kvr
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        kvr.query_rope(z(2, 1, 64), i, z(2, 1, 64))
    with pytest.raises(ValueError):
        kvr.kv_cache_read(z(1, 2, 1, 8), z(1, 2, 1, 8), i, z(2, 16))
    with pytest.raises(ValueError):
        kvr.mla_attention(z(1, 1, 512), z(1, 1, 64), z(1, 2, 1, 512), z(1, 2, 1, 64), i.view(1, 2), i, i[:1], z(1, 1, 512), softmax_scale=1.0)
    with pytest.raises(TypeError):
        kvr.query_rope(None, i, None)
