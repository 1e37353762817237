"""Oracle for the operators around the cache: the query's RoPE with several
axes, reading cache rows back, and latent attention over the caches.

Test infrastructure only (see oracle/__init__.py). float64 NumPy, written from
the definitions:

* query_rope: "aclnnMlaPrologV3WeightNz", "Formula" (q^R = ROPE(...)), by
  "aclnnKvRmsNormRopeCache", "Formulas (1) interleaveRope", angle of pair i =
  position on its axis times base^(-2i/D);
* cache rows: "aclnnKvRmsNormRopeCache", "Restrictions on index"; an 8-bit code
  stands for code / scale ("Restrictions on quantization scenarios", where the
  code written is round(value * scale));
* attention: softmax(scale * (q_nope . c + q_rope . k)) c over the keys that a
  token sees.
"""
import numpy as np

from .kv_rmsnorm_rope_cache import cache_slot

STATUS_QUERY = 0x20
STATUS_KEY_LENGTH = 0x2
STATUS_INDEX = 0x1


def rope_angles(positions, sections, D, base):
    """Angles [T, D/2] of int positions [axes, T]."""
    axis = np.repeat(np.arange(len(sections)), sections)
    inv = float(base) ** (-2.0 * np.arange(D // 2) / D)
    return np.asarray(positions, dtype=np.float64)[axis].T * inv


def ref_query_rope(q, positions, sections, base=10000.0, half_pairs=False):
    """q float64 [T, H, D] -> (out [T, H, D], cos [T, D], sin [T, D])."""
    D = q.shape[-1]
    ang = rope_angles(positions, sections, D, base)
    c, s = np.cos(ang), np.sin(ang)
    a, b = (q[..., :D // 2], q[..., D // 2:]) if half_pairs else (q[..., 0::2], q[..., 1::2])
    cc, ss = c[:, None], s[:, None]
    out = np.concatenate([a * cc - b * ss, b * cc + a * ss], axis=-1)
    return out, np.concatenate([c, c], -1), np.concatenate([s, s], -1)


def ref_kv_cache_read(out, ckv, k, index, mode, ckv_scale=None, k_scale=None):
    """out float64 [B, S, Dv + Dk] (changed in place), caches float64 values of
    the codes [d0, d1, D*]. Returns the status bits."""
    B, S = out.shape[:2]
    d0, d1, Dv = ckv.shape
    status = 0
    for b in range(B):
        for s in range(S):
            slot = cache_slot(mode, b, s, index, S, d0, d1)
            if isinstance(slot, tuple):
                c, r = ckv[slot], k[slot]
                out[b, s, :Dv] = c if ckv_scale is None else c / ckv_scale
                out[b, s, Dv:] = r if k_scale is None else r / k_scale
            elif slot == "bad":
                status |= STATUS_INDEX
    return status


def ref_mla_attention(q_nope, q_rope, ckv, k, table, query_start, key_length, out, lse, *, scale, causal=True,
                      ckv_scale=None, k_scale=None):
    """float64 arrays: q_nope [T, H, Dv], q_rope [T, H, Dk], caches [d0, d1, D*]
    of code values, out [T, H, Dv] and lse [T, H] changed in place. table int
    [N, blocks], or None where sequence n reads cache batch n.

    Returns (status, A, B): for each output row the weights' sum of magnitudes
    A[t, h, c] = sum_i p_i |c_i| and the size of its largest score's terms
    B[t, h] = scale * max_i sum |q||key|, which bound what rounding can do."""
    d0, d1 = ckv.shape[:2]
    T = q_nope.shape[0]
    A, B = np.zeros(out.shape), np.zeros(lse.shape)
    status = 0
    most = d1 if table is None else table.shape[1] * d1
    for n in range(len(key_length)):
        a, b, K = int(query_start[n]), int(query_start[n + 1]), int(key_length[n])
        if a < 0 or b < a or b > T:
            status |= STATUS_QUERY
            continue
        if a == b:
            continue
        if K < 0 or K > most:
            status |= STATUS_KEY_LENGTH
            continue
        i = np.arange(K)
        if table is None:
            at = np.stack([np.full(K, n), i], -1)
            live = np.ones(K, bool)
        else:
            e = np.asarray(table[n], dtype=np.int64)[i // d1] if K else np.zeros(0, np.int64)
            live = (e >= 0) & (e < d0)
            at = np.stack([e, i % d1], -1)
        if np.any(~live & (at[:, 0] != -1)):   # the sequence's last token sees all K keys
            status |= STATUS_INDEX
        keys = i[live]
        c = ckv[at[live, 0], at[live, 1]]
        r = k[at[live, 0], at[live, 1]]
        c = c if ckv_scale is None else c / ckv_scale
        r = r if k_scale is None else r / k_scale
        for t in range(a, b):
            sees = K - (b - 1 - t) if causal else K
            vis = keys < sees
            if not vis.any():
                out[t], lse[t] = 0.0, -np.inf
                continue
            cv, rv = c[vis], r[vis]
            s = scale * (q_nope[t] @ cv.T + q_rope[t] @ rv.T)
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            out[t] = p @ cv / l
            lse[t] = (m + np.log(l))[:, 0]
            A[t] = p @ np.abs(cv) / l
            B[t] = abs(scale) * (np.abs(q_nope[t]) @ np.abs(cv).T + np.abs(q_rope[t]) @ np.abs(rv).T).max(-1)
    return status, A, B
