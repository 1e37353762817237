"""Cases, oracle runs and tolerances for query_rope, kv_cache_read and mla_attention."""
from dataclasses import dataclass

import numpy as np
import torch

from helpers import f64, guarded

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.int8, "fp8_e4m3fn": torch.float8_e4m3fn,
          "fp8_e5m2": torch.float8_e5m2}


def half_step(dtype):
    """Largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def cache_values(g, shape, dtype, scale_len=None):
    """(cache tensor, float32 scale or None): N(0, 1) values, or codes of value * scale."""
    x = torch.randn(shape, generator=g)
    if dtype in ("bf16", "f16"):
        return x.to(DTYPES[dtype]), None
    s = torch.rand(scale_len, generator=g) * 1.5 + 0.5
    if dtype == "int8":
        s = s * 20
        return (x * s).round().clamp(-128, 127).to(torch.int8), s
    return (x * s).to(DTYPES[dtype]), s


@dataclass
class MlaCase:
    q_nope: torch.Tensor
    q_rope: torch.Tensor
    ckv: torch.Tensor
    k: torch.Tensor
    ckv_scale: torch.Tensor
    k_scale: torch.Tensor
    table: torch.Tensor
    query_start: torch.Tensor
    key_length: torch.Tensor
    scale: float
    causal: bool
    mode: str


def mla_case(new, keys, H=4, Dv=512, Dk=64, block_size=16, dtype="bf16", cache=None, k_cache=None, scale_len=1, k_scale_len=1,
             seed=0, causal=True, mode="PA_BSND", gap=0, holes=(), scale=0.0722, spread=1.0, pad=0):
    """new, keys: per sequence. gap: rows of q behind the last sequence. holes:
    (sequence, block) entries set to -1. pad: extra channels in front of each
    q row (strided rows). Cache rows that no key names are NaN."""
    g = torch.Generator().manual_seed(seed)
    N, T = len(new), sum(new) + gap
    cache, k_cache = cache or dtype, k_cache or dtype
    nan = lambda t: t.view(torch.int16).fill_(0x7FFF) if t.element_size() == 2 else t.view(torch.uint8).fill_(0x7F)  # noqa: E731
    table = None
    if mode == "Norm":
        d0, d1 = N + 1, max(max(keys), 1) + 3
        slots = [n * d1 + torch.arange(keys[n]) for n in range(N)]
    else:
        d1 = block_size
        pages = [-(-x // d1) for x in keys]
        d0 = sum(pages) + 2
        order = torch.randperm(d0, generator=g)
        table = torch.full((N, max(pages + [1]) + 1), -1, dtype=torch.int64)
        at, slots = 0, []
        for n in range(N):
            table[n, :pages[n]] = order[at:at + pages[n]]
            at += pages[n]
            i = torch.arange(keys[n])
            slots.append(table[n, i // d1] * d1 + i % d1)
    ckv, cs = cache_values(g, (d0 * d1, Dv), cache, Dv if scale_len != 1 else 1)
    k, ks = cache_values(g, (d0 * d1, Dk), k_cache, Dk if k_scale_len != 1 else 1)
    used = torch.zeros(d0 * d1, dtype=torch.bool)
    if slots:
        used[torch.cat(slots)] = True
    for t in (ckv, k):   # int8 has no NaN: 127 stands in
        blank = torch.empty_like(t)
        nan(blank)
        t.view(torch.int16 if t.element_size() == 2 else torch.uint8)[~used] = \
            blank.view(torch.int16 if t.element_size() == 2 else torch.uint8)[~used]
    for n, b in holes:
        table[n, b] = -1
    qw = (torch.randn(T, H, pad + Dv + Dk, generator=g) * spread).to(DTYPES[dtype])
    start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int64)
    return MlaCase(qw[..., pad:pad + Dv], qw[..., pad + Dv:], ckv.view(d0, d1, 1, Dv), k.view(d0, d1, 1, Dk), cs, ks, table,
                   start, torch.tensor(keys, dtype=torch.int64), scale, causal, mode)


SENTINEL = -77.0


def on_tensor_cores(c):
    """Whether the call takes the tensor-core kernel, which alone needs a workspace."""
    import attention_prologue_kv_gb300 as kvr
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    call = kvr.prepare_mla_attention(c.q_nope.cuda(), c.q_rope.cuda(), d(c.ckv), d(c.k), d(c.table), d(c.query_start),
                                     d(c.key_length), torch.empty_like(c.q_nope, device="cuda").contiguous(),
                                     softmax_scale=c.scale, cache_mode=c.mode, ckv_scale=d(c.ckv_scale), k_scale=d(c.k_scale))
    return call.workspace is not None


def run_mla(c, workspace=None, stream=None, lse=True):
    """(out float64, lse float64, status) of the GPU call; untouched rows hold SENTINEL."""
    import attention_prologue_kv_gb300 as kvr
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    T, H, Dv = c.q_nope.shape
    out, c1 = guarded((T, H, Dv), c.q_nope.dtype, SENTINEL)
    ls, c2 = guarded((T, H), torch.float32, SENTINEL)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = c.q_nope._base
    if wide is not None and wide.shape[-1] != Dv:   # keep the strided rows
        w = wide.cuda()
        lo = c.q_nope.storage_offset()
        qn, qr = w[..., lo:lo + Dv], w[..., lo + Dv:lo + Dv + c.q_rope.shape[-1]]
    else:
        qn, qr = c.q_nope.cuda(), c.q_rope.cuda()
    kvr.mla_attention(qn, qr, d(c.ckv), d(c.k), d(c.table), d(c.query_start), d(c.key_length), out, softmax_scale=c.scale,
                      cache_mode=c.mode, causal=c.causal, ckv_scale=d(c.ckv_scale), k_scale=d(c.k_scale),
                      lse=ls if lse else None, dev_status=st, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    c1()
    c2()
    return f64(out), f64(ls), int(st.item())


def oracle_mla(c, q_nope=None, q_rope=None):
    import oracle
    T, H, Dv = c.q_nope.shape
    out, lse = np.full((T, H, Dv), SENTINEL), np.full((T, H), SENTINEL)
    n = lambda t: None if t is None else t.numpy()  # noqa: E731
    with np.errstate(invalid="ignore", over="ignore"):
        st, A, B = oracle.ref_mla_attention(
            f64(c.q_nope) if q_nope is None else q_nope, f64(c.q_rope) if q_rope is None else q_rope, f64(c.ckv)[:, :, 0],
            f64(c.k)[:, :, 0], n(c.table), n(c.query_start), n(c.key_length), out, lse, scale=float(np.float32(c.scale)),
            causal=c.causal, ckv_scale=None if c.ckv_scale is None else f64(c.ckv_scale),
            k_scale=None if c.k_scale is None else f64(c.k_scale))
    return out, lse, st, A, B


def rounded_query(c):
    """q as the tensor-core kernel multiplies it where a cache has a scale per
    channel, in float64: the latent part as halves of q / scale, over a power of two
    per row (of its largest |q| and the largest 1 / scale) that keeps them below
    2^14; the rotary part as q / scale in q's type, a power of two over the
    largest 1 / scale taken out."""
    def inverse(s):
        return (1.0 / s).to(torch.float32)

    n64, r64 = f64(c.q_nope), f64(c.q_rope)
    if c.ckv_scale is not None and c.ckv_scale.numel() > 1:
        inv = inverse(c.ckv_scale)
        q = c.q_nope.to(torch.float32)
        x = q * inv
        g = 2.0 ** (13 - torch.floor(torch.log2(q.abs().amax(-1, keepdim=True))) - torch.ceil(torch.log2(inv.max())))
        n64 = f64((x * g).to(torch.float16)) / f64(g) * f64(c.ckv_scale)
    if c.k_scale is not None and c.k_scale.numel() > 1:
        lift = 2.0 ** torch.ceil(torch.log2(inverse(c.k_scale).max()))
        r64 = f64((c.q_rope.to(torch.float32) * (inverse(c.k_scale) / lift)).to(c.q_rope.dtype)) * f64(c.k_scale) * float(lift)
    return n64, r64


def check_mla(c, gpu, ref, p_rounded=True):
    """Bounds, to first order, with u = half a step of the type:
    * a score is a sum of at most 576 + products in float32: 16 at a time on the
      tensor cores or 18 chained plus 5 butterfly adds on the plain kernel, at
      most 64 roundings of 2^-23 of the terms' size B: |ds| <= 2^-17 B (the
      exponential and the scale add 2^-21 (1 + |s|), which 2^-17 B + 2^-19 covers);
    * a weight is off by the factor e^(2 ds) after the division: 2 |ds| A;
    * rounding each weight to the type moves the sum by at most u A (tensor-core kernel);
    * the float32 sums over n keys: n 2^-23 A;
    * the output's own rounding: u |out|.
    lse moves by |ds| + n 2^-23, and is stored in float32."""
    out, lse, st = gpu
    rout, rlse, rst, A, B = ref
    assert st == rst
    u = half_step(c.q_nope.dtype)
    n = int(c.key_length.max()) if c.key_length.numel() else 0
    ds = 2.0 ** -17 * B + 2.0 ** -19
    rel = 2 * ds[..., None] + (u if p_rounded else 0.0) + n * 2.0 ** -23 + 2.0 ** -20
    tiny = float(torch.finfo(c.q_nope.dtype).tiny) * 2.0 ** -3
    tol = u * np.abs(rout) + rel * A * (1 + u) + tiny
    bad = ~(np.abs(out - rout) <= tol)
    assert not bad.any(), "%d of %d outputs out of bounds, e.g. gpu %s ref %s tol %s at %s" % (
        bad.sum(), bad.size, out[bad][:3], rout[bad][:3], tol[bad][:3], np.argwhere(bad)[:3].tolist())
    fin = np.isfinite(rlse)
    assert np.array_equal(lse[~fin], rlse[~fin])
    off = np.abs(lse[fin] - rlse[fin]) - ds[fin] - n * 2.0 ** -23 - 2.0 ** -23 * np.abs(rlse[fin])
    assert not (off > 0).any(), "lse off by %g more than its bound" % off.max()
    return float(np.abs(out - rout).max() / max(1e-30, np.abs(rout).max()))
