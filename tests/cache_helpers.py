"""Cases, oracle runs and tolerances for drafted trees, key weights, selection and compaction."""
import numpy as np
import torch

from attention_helpers import MlaCase, SENTINEL, mla_case, oracle_mla
from helpers import f64, guarded


def parents(counts, seed, chain=False):
    """int64 [T]: each first token continues the context, every other a token before it (some the context too)."""
    r = np.random.default_rng(seed)
    out = []
    for n in counts:
        out += [-1 if j == 0 or (not chain and r.random() < 0.1) else (j - 1 if chain else int(r.integers(0, j))) for j in range(n)]
    return torch.tensor(out, dtype=torch.int64)


def tree_words(c: MlaCase, words, seed, chain=False):
    """int64 [T, words] by the oracle: ancestors in random trees over a case's new tokens."""
    import oracle
    start = c.query_start.numpy()
    mask = np.zeros((c.q_nope.shape[0], words), dtype=np.int64)
    up = parents(list(start[1:] - start[:-1]), seed, chain).numpy()
    up = np.concatenate([up, np.full(c.q_nope.shape[0] - len(up), -1)])
    oracle.ref_draft_tree(up, start, mask)
    return torch.from_numpy(mask)


def cuda(t):
    return None if t is None else t.cuda()


def queries(c):
    """q_nope and q_rope on the GPU, strided rows kept."""
    Dv, wide = c.q_nope.shape[-1], c.q_nope._base
    if wide is None or wide.shape[-1] == Dv:
        return c.q_nope.cuda(), c.q_rope.cuda()
    w, lo = wide.cuda(), c.q_nope.storage_offset()
    return w[..., lo:lo + Dv], w[..., lo + Dv:lo + Dv + c.q_rope.shape[-1]]


def run_tree(c, mask, stream=None, workspace=None):
    import attention_prologue_kv_gb300 as kvr
    T, H, Dv = c.q_nope.shape
    out, c1 = guarded((T, H, Dv), c.q_nope.dtype, SENTINEL)
    ls, c2 = guarded((T, H), torch.float32, SENTINEL)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.mla_attention(*queries(c), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length), out,
                      softmax_scale=c.scale, cache_mode=c.mode, ckv_scale=cuda(c.ckv_scale), k_scale=cuda(c.k_scale), lse=ls,
                      dev_status=st, tree_mask=mask.cuda(), stream=stream, workspace=workspace)
    torch.cuda.synchronize()
    c1()
    c2()
    return f64(out), f64(ls), int(st.item())


def oracle_tree(c, mask, q_nope=None, q_rope=None):
    import oracle
    T, H, Dv = c.q_nope.shape
    out, lse = np.full((T, H, Dv), SENTINEL), np.full((T, H), SENTINEL)
    n = lambda t: None if t is None else t.numpy()  # noqa: E731
    with np.errstate(invalid="ignore", over="ignore"):
        st, A, B = oracle.ref_mla_tree_attention(
            f64(c.q_nope) if q_nope is None else q_nope, f64(c.q_rope) if q_rope is None else q_rope, f64(c.ckv)[:, :, 0],
            f64(c.k)[:, :, 0], n(c.table), n(c.query_start), n(c.key_length), mask.numpy(), out, lse,
            scale=float(np.float32(c.scale)), ckv_scale=None if c.ckv_scale is None else f64(c.ckv_scale),
            k_scale=None if c.k_scale is None else f64(c.k_scale))
    return out, lse, st, A, B


def row_lse(c):
    """float32 [T, H]: what attention over the case's keys gives, by the oracle; 0 in rows outside every sequence."""
    lse = oracle_mla(c)[1]
    return torch.from_numpy(np.where(lse == SENTINEL, 0.0, lse)).to(torch.float32)


def run_weight(c, lse, width, past=None, decay=1.0, in_place=False, pad=0, stream=None, workspace=None):
    """(weight float64 [N, width], status): untouched entries hold SENTINEL. past: float32 [N, width] or None. pad: entries
    between the rows."""
    import attention_prologue_kv_gb300 as kvr
    N = len(c.key_length)
    wide, check = guarded((N, width + pad), torch.float32, SENTINEL)
    w = wide[:, :width]
    old = None if past is None else past.cuda()
    if in_place:
        w.copy_(past)
        old = w
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.mla_key_weight(*queries(c), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length), lse.cuda(), w,
                       softmax_scale=c.scale, cache_mode=c.mode, causal=c.causal, past=old, decay=decay,
                       ckv_scale=cuda(c.ckv_scale), k_scale=cuda(c.k_scale), dev_status=st, stream=stream, workspace=workspace)
    torch.cuda.synchronize()
    check()
    assert pad == 0 or bool((wide[:, width:] == SENTINEL).all())
    return f64(w), int(st.item())


def oracle_weight(c, lse, width, past=None, decay=1.0, in_place=False):
    import oracle
    N = len(c.key_length)
    w = np.full((N, width), SENTINEL) if not in_place else f64(past)
    n = lambda t: None if t is None else t.numpy()  # noqa: E731
    with np.errstate(invalid="ignore", over="ignore"):
        st, E, rows = oracle.ref_mla_key_weight(
            f64(c.q_nope), f64(c.q_rope), f64(c.ckv)[:, :, 0], f64(c.k)[:, :, 0], n(c.table), n(c.query_start), n(c.key_length),
            f64(lse), w, scale=float(np.float32(c.scale)), causal=c.causal, past=None if past is None else f64(past),
            decay=float(np.float32(decay)), ckv_scale=None if c.ckv_scale is None else f64(c.ckv_scale),
            k_scale=None if c.k_scale is None else f64(c.k_scale))
    return w, st, E, rows


def check_weight(c, gpu, ref, past=None, decay=1.0):
    """Bounds, to first order:
    * a score is a sum of at most 576 + products in float32, at most 64 roundings of 2^-23 of the terms' size B each (16
      products an addition on the tensor cores, 18 chained and 5 butterfly adds on the plain kernel). A query divided by a
      scale per channel is held as the sum of two halves: 22 bits of it, 2^-22 B more; the rotary part beside latent codes with
      one scale as two parts of its type, 2^-18 B more at most (bf16). With lse in the exponent, and its and the
      score's product with log2 e: |d(s - lse)| <= 2^-17 B + 2^-21 (1 + |s| + |lse|) <= 2^-17 (B + 1 + |s| + |lse|);
    * a weight is off by that factor: 2^-17 E; to second order 2^-16 E covers it;
    * the float32 sum over r rows: r 2^-24 of the sum at most, and the exponential itself 2^-21;
    * decay * past: its own rounding and that of the sum, 2^-23 of each."""
    w, st = gpu
    rw, rst, E, rows = ref
    assert st == rst
    old = np.zeros(rw.shape) if past is None else np.abs(decay * f64(past))
    tol = 2.0 ** -16 * E + (rows[:, None] * 2.0 ** -24 + 2.0 ** -21) * np.abs(rw) + 2.0 ** -22 * old + 2.0 ** -120
    bad = ~(np.abs(w - rw) <= tol)
    assert not bad.any(), "%d of %d weights out of bounds, e.g. gpu %s ref %s tol %s at %s" % (
        bad.sum(), bad.size, w[bad][:3], rw[bad][:3], tol[bad][:3], np.argwhere(bad)[:3].tolist())


__all__ = ["mla_case"]
