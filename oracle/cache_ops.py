"""Oracle for drafted trees and caches of bounded size: ancestors of drafted
tokens, latent attention of a tree, the attention weight of each key, which keys
to keep, and moving kept rows together.

Test infrastructure only (see oracle/__init__.py). NumPy, float64 where values
are computed, written from the definitions in include/kvr.h.
"""
import numpy as np

from .attention_step import STATUS_INDEX, STATUS_KEY_LENGTH, STATUS_QUERY


def ancestors(parent):
    """Sets of places, the token's own among them, from a sequence's parents."""
    out = []
    for j, up in enumerate(parent):
        out.append((set(out[up]) if 0 <= up < j else set()) | {j})
    return out


def ref_draft_tree(parent, query_start, mask, position_start=None, positions=None):
    """mask int64 [T, words] and positions int64 [T] changed in place. Returns the status bits."""
    T, words = mask.shape
    status = 0
    for n in range(len(query_start) - 1):
        a, b = int(query_start[n]), int(query_start[n + 1])
        if a < 0 or b < a or b > T or b - a > 64 * words:
            status |= STATUS_QUERY
            continue
        ups = [int(x) for x in parent[a:b]]
        if any(not -1 <= x < j for j, x in enumerate(ups)):
            status |= STATUS_INDEX
        for j, places in enumerate(ancestors(ups)):
            word = [0] * words
            for x in places:
                word[x // 64] |= 1 << (x % 64)
            mask[a + j] = np.array(word, dtype=np.uint64).view(np.int64)
            if positions is not None:
                positions[a + j] = int(position_start[n]) + len(places) - 1
    return status


def _bits(words):
    return {64 * w + b for w, x in enumerate(np.asarray(words).astype(np.int64).view(np.uint64)) for b in range(64) if int(x) >> b & 1}


def steps(T, d0, d1, table, query_start, key_length, most_new, most_keys):
    """(status, [(n, first row, end row, keys' places, their cache rows)]) of the sequences that are not left out."""
    status, out = 0, []
    most = d1 if table is None else table.shape[1] * d1
    for n in range(len(key_length)):
        a, b, K = int(query_start[n]), int(query_start[n + 1]), int(key_length[n])
        if a < 0 or b < a or b > T or b - a > most_new:
            status |= STATUS_QUERY
            continue
        if a == b:
            continue
        if K < 0 or K > min(most, most_keys):
            status |= STATUS_KEY_LENGTH
            continue
        i = np.arange(K)
        e = np.full(K, n) if table is None else np.asarray(table[n], dtype=np.int64)[i // d1]
        r = i if table is None else i % d1
        live = (e >= 0) & (e < d0)
        if np.any(~live & (e != -1)):
            status |= STATUS_INDEX
        out.append((n, a, b, K, i[live], (e[live], r[live])))
    return status, out


def sees(keys, K, L, j, causal, words=None):
    """Which of the places `keys` token j of L sees."""
    if words is not None:
        bits = _bits(words)
        return np.array([x < K - L or (x - (K - L)) in bits for x in keys], dtype=bool)
    return keys < (K - L + j + 1 if causal else K)


def _scores(qn, qr, c, r, scale):
    return scale * (qn @ c.T + qr @ r.T), abs(scale) * (np.abs(qn) @ np.abs(c).T + np.abs(qr) @ np.abs(r).T)


def _rows(ckv, k, at, ckv_scale, k_scale):
    c, r = ckv[at], k[at]
    return (c if ckv_scale is None else c / ckv_scale), (r if k_scale is None else r / k_scale)


def ref_mla_tree_attention(q_nope, q_rope, ckv, k, table, query_start, key_length, mask, out, lse, *, scale, ckv_scale=None,
                           k_scale=None):
    """As ref_mla_attention, with mask int64 [T, words]."""
    d0, d1 = ckv.shape[:2]
    A, B = np.zeros(out.shape), np.zeros(lse.shape)
    status, todo = steps(q_nope.shape[0], d0, d1, table, query_start, key_length, 64 * mask.shape[1], 1 << 24)
    for n, a, b, K, keys, at in todo:
        c, r = _rows(ckv, k, at, ckv_scale, k_scale)
        for t in range(a, b):
            vis = sees(keys, K, b - a, t - a, False, mask[t])
            if not vis.any():
                out[t], lse[t] = 0.0, -np.inf
                continue
            s, size = _scores(q_nope[t], q_rope[t], c[vis], r[vis], scale)
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            out[t] = p @ c[vis] / l
            lse[t] = (m + np.log(l))[:, 0]
            A[t] = p @ np.abs(c[vis]) / l
            B[t] = size.max(-1)
    return status, A, B


def ref_mla_key_weight(q_nope, q_rope, ckv, k, table, query_start, key_length, lse, weight, *, scale, causal=True, past=None,
                       decay=1.0, ckv_scale=None, k_scale=None):
    """weight float64 [N, width] changed in place. Returns (status, E, rows): E [N, width] bounds what an error of a unit
    in the terms of a score and of lse does to the weight, sum p (B + 1 + |s| + |lse|) with B the sum of a score's terms'
    magnitudes; rows [N] how many terms a weight has."""
    d0, d1 = ckv.shape[:2]
    E, rows = np.zeros(weight.shape), np.zeros(len(key_length))
    old = None if past is None else np.array(past, dtype=np.float64)
    status, todo = steps(q_nope.shape[0], d0, d1, table, query_start, key_length, q_nope.shape[0], min(weight.shape[1], 1 << 24))
    for n, a, b, K, keys, at in todo:
        c, r = _rows(ckv, k, at, ckv_scale, k_scale)
        weight[n, :K] = 0 if old is None else decay * old[n, :K]
        rows[n] = (b - a) * q_nope.shape[1]
        for t in range(a, b):
            vis = sees(keys, K, b - a, t - a, causal)
            if not vis.any():
                continue
            s, size = _scores(q_nope[t], q_rope[t], c[vis], r[vis], scale)
            live = lse[t] != -np.inf
            p = np.exp(s[live] - lse[t][live, None])
            weight[n, keys[vis]] += p.sum(0)
            terms = size[live] + 1 + np.abs(s[live]) + np.abs(lse[t][live, None])
            E[n, keys[vis]] += np.where(p == 0, 0.0, p * terms).sum(0)   # (0 where lse is infinite)
    return status, E, rows


def ref_kv_cache_select(weight, key_length, keep, sink=0, recent=0):
    """(status, kept [N, keep], kept_length [N], kept weights [N, keep]) by sorting."""
    n, width = weight.shape
    kept, count, carried = np.full((n, keep), -1, dtype=np.int64), np.zeros(n, dtype=np.int64), np.zeros((n, keep), weight.dtype)
    status = 0
    for i in range(n):
        K = int(key_length[i])
        if K < 0 or K > width:
            status |= STATUS_KEY_LENGTH
            continue
        if K <= keep:
            mine = list(range(K))
        else:
            w = [float(x) for x in weight[i, :K]]
            between = sorted(range(sink, K - recent), key=lambda x: (0, 0.0, x) if np.isnan(w[x]) else (1, -w[x], x))
            mine = sorted(list(range(sink)) + list(range(K - recent, K)) + between[:keep - sink - recent])
        kept[i, :len(mine)] = mine
        carried[i, :len(mine)] = weight[i, mine]
        count[i] = len(mine)
    return status, kept, count, carried


def ref_kv_cache_compact(ckv, k, table, kept, kept_length, start=None):
    """ckv, k [d0, d1, D*] changed in place (any type). Returns the status bits."""
    d0, d1 = ckv.shape[:2]
    most = d1 if table is None else table.shape[1] * d1
    status = 0
    for n in range(len(kept_length)):
        count, first = int(kept_length[n]), 0 if start is None else int(start[n])
        if count < 0 or count > kept.shape[1] or first < 0 or first + count > most:
            status |= STATUS_KEY_LENGTH
            continue
        place = lambda x: (n, x) if table is None else (int(table[n][x // d1]), x % d1)  # noqa: E731,B023
        moves = []
        for i in range(count):
            of, before = int(kept[n, i]), int(kept[n, i - 1]) if i else -1
            if not (of > before and of >= first + i and of < most):
                status |= STATUS_INDEX
            elif of != first + i:
                x, y = place(of), place(first + i)
                if 0 <= x[0] < d0 and 0 <= y[0] < d0:
                    moves.append((y, ckv[x].copy(), k[x].copy()))
                else:
                    status |= STATUS_INDEX
        for y, c, r in moves:
            ckv[y], k[y] = c, r
    return status
