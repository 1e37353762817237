"""What is measured of the operators beside the KV prologue: attention over the latent cache
(`mla_attention`), reading cache rows back (`kv_cache_read`) and the rotary positions of the query
with several axes (`query_rope`), each in plain torch operations and as the library's call.

The head split is the one of the repository's workloads: Dv = 512 latent channels and Dk = 64
rotary channels, one key row per token for all heads.
"""
import random

import torch

own = False

DV, DK = 512, 64
SOFTMAX_SCALE = 0.0722   # scores of N(0, 1) queries and keys then spread over about +-5, as trained heads do
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.int8,
          "fp8_e4m3fn": torch.float8_e4m3fn, "fp8_e5m2": torch.float8_e5m2}


def listed():
    return [
        # one conversation answered alone on one of eight cards that share the heads: latency
        attention_case("attn_decode_one", seqs=1, new=(1, 1), keys=(1000, 1000), heads=16, lengths=1),
        # a decode step of a full batch, every head on this card, contexts of all ages
        attention_case("attn_decode_batch", seqs=256, new=(1, 1), keys=(1, 4095), heads=128, lengths=2),
        # the same with the latent part of the cache in 8 bits, longer contexts, fewer sequences
        attention_case("attn_decode_fp8", seqs=61, new=(1, 1), keys=(3000, 16384), heads=128, cache="fp8_e4m3fn",
                       scale="channel", lse=False, lengths=3),
        # drafted tokens checked in one step: a few new tokens per sequence, small pages, int8, few heads
        attention_case("attn_draft_int8", seqs=33, new=(1, 7), keys=(7, 2500), heads=20, dtype="f16", cache="int8",
                       scale="tensor", block_size=16, lengths=4),
        # chunks of several prompts beside each other
        attention_case("attn_chunk_mixed", seqs=8, new=(33, 129), keys=(200, 4096), heads=128, lengths=5),
        # one chunk of a long prompt: the largest
        attention_case("attn_chunk_long", seqs=1, new=(512, 512), keys=(16384, 16384), heads=128, lengths=6),
        # the rows of a decode batch read back at their slots, some of them skipped
        read_case("read_decode", seqs=256, tokens=1, mode="PA_BSND", skip=5),
        # the context of a chunk read back from an 8-bit cache by blocks, for the form that expands the heads
        read_case("read_context_fp8", seqs=8, tokens=4096, mode="PA_BLK_BSND", cache="fp8_e4m3fn", scale="channel"),
        # odd lengths, one cache batch per sequence, both parts in int8
        read_case("read_norm_int8", seqs=37, tokens=531, mode="Norm", block_size=1031, cache="int8", k_cache="int8",
                  scale="channel", skip=400),
        # a decode batch's queries, one axis, the tables for the prologue written beside
        rope_case("rope_decode", tokens=256, heads=128, axes=1),
        # a prompt with images: time, height and width, the queries a slice of a wider projection
        rope_case("rope_image_prompt", tokens=8191, heads=128, axes=3, wide=128),
    ]


def attention_case(name, seqs, new, keys, heads, lengths, dtype="bf16", cache="bf16", scale="none", block_size=128,
                   lse=True):
    c = {"op": "attention", "seqs": seqs, "new_min": new[0], "new_max": new[1], "keys_min": keys[0], "keys_max": keys[1],
         "heads": heads, "lengths": lengths, "dtype": dtype, "cache": cache, "scale": scale, "block_size": block_size,
         "lse": lse}
    return dict(c, name=name) if name else c


def read_case(name, seqs, tokens, mode, dtype="bf16", cache="bf16", k_cache="bf16", scale="none", block_size=128, skip=0):
    c = {"op": "read", "seqs": seqs, "tokens": tokens, "mode": mode, "dtype": dtype, "cache": cache, "k_cache": k_cache,
         "scale": scale, "block_size": block_size, "skip": skip}
    return dict(c, name=name) if name else c


def rope_case(name, tokens, heads, axes, dtype="bf16", dim=DK, wide=0, layout="interleave", tables=True):
    c = {"op": "rope", "tokens": tokens, "heads": heads, "axes": axes, "dtype": dtype, "dim": dim, "wide": wide,
         "layout": layout, "tables": tables}
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["attention", "attention", "read", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([dtype, dtype, "int8", "fp8_e4m3fn", "fp8_e5m2"])
    scale = "none" if cache == dtype else rng.choice(["channel", "tensor"])
    if op == "attention":
        heads = _log_int(rng, 1, 128)
        most_new = _log_int(rng, 1, 512)
        most_keys = _log_int(rng, max(8, most_new), 16384)
        # at most about the rows x keys of the largest listed case, and as many keys as the largest decode batch
        seqs = max(1, min(_log_int(rng, 1, 256), 500000000 // (most_new * heads * most_keys), 600000 // most_keys))
        return attention_case(None, seqs, (rng.randint(1, most_new), most_new), (rng.randint(1, most_keys), most_keys), heads,
                              rng.randint(1, 10 ** 6), dtype, cache, scale, rng.choice([16, 32, 64, 100, 128, 256]),
                              scale != "channel")
    if op == "read":
        seqs = _log_int(rng, 1, 256)
        tokens = min(_log_int(rng, 1, 4096), 32768 // seqs)
        mode = rng.choice(["PA_BSND", "PA_BLK_BSND", "Norm"])
        block = rng.randint(tokens, tokens + 500) if mode == "Norm" else rng.choice([16, 33, 64, 128])
        k_cache = dtype if scale == "none" or rng.random() < 0.5 else cache
        return read_case(None, seqs, tokens, mode, dtype, cache, k_cache, scale, block,
                         rng.randint(0, seqs) if mode != "PA_BLK_BSND" else 0)
    heads = _log_int(rng, 1, 128)
    tokens = _log_int(rng, 1, min(32768, 1048448 // heads))
    dim = rng.choice([32, 64, 64, 128])
    tokens = max(1, tokens * 64 // dim if dim > 64 else tokens)
    return rope_case(None, tokens, heads, rng.choice([1, 2, 3, 4]), dtype, dim, rng.choice([0, 0, 128]),
                     rng.choice(["interleave", "half"]), rng.random() < 0.7)


def _lengths(c):
    """New tokens and keys (the new ones among them) of each sequence; the case's own, whatever the seed."""
    r = random.Random(c["lengths"])
    new = [r.randint(c["new_min"], c["new_max"]) for _ in range(c["seqs"])]
    keys = [max(n, r.randint(c["keys_min"], c["keys_max"])) for n in new]
    return new, keys


def _row_bytes(c):
    size = {"bf16": 2, "f16": 2}
    return DV * size.get(c["cache"], 1) + DK * size.get(c.get("k_cache", "bf16"), 1)


def work(c):
    if c["op"] == "attention":
        new, keys = _lengths(c)
        pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(new, keys))   # (token, key) pairs that the causal mask leaves
        rows = sum(new) * c["heads"]
        pages = sum(-(-k // c["block_size"]) for k in keys)
        scales = {"none": 0, "tensor": 4, "channel": 4 * DV}[c["scale"]]
        return {"bytes": rows * (DV + DK + DV) * 2 + sum(keys) * _row_bytes(c) + 8 * (pages + 2 * len(keys) + 1) + scales
                + (4 * rows if c["lse"] else 0),
                "flops": 2 * pairs * c["heads"] * (DV + DK + DV)}
    if c["op"] == "read":
        rows = c["seqs"] * c["tokens"]
        entries = c["seqs"] * -(-c["tokens"] // c["block_size"]) if c["mode"] == "PA_BLK_BSND" else rows
        live = rows - c["skip"]
        return {"bytes": live * (_row_bytes(c) + (DV + DK) * 2) + 8 * entries, "flops": live * (DV + DK)}
    rows, d = c["tokens"] * c["heads"], c["dim"]
    return {"bytes": rows * d * 4 + 8 * c["axes"] * c["tokens"] + (c["tokens"] * d * 4 if c["tables"] else 0),
            "flops": rows * d * 3}


def _cache_part(gen, rows, width, dtype, scale):
    """Rows of one part of a cache as the prologue leaves them: about N(0, 1) values, or the codes of value * scale."""
    x = torch.randn(rows, width, generator=gen, device="cuda", dtype=torch.float32)
    if dtype in ("bf16", "f16"):
        return x.to(DTYPES[dtype]), None
    s = torch.rand(width if scale == "channel" else 1, generator=gen, device="cuda") * 1.5 + 0.5
    if dtype == "int8":
        s = s * 20
        return (x * s).round().clamp(-128, 127).to(torch.int8), s
    return (x * s).to(DTYPES[dtype]), s


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "read": _prepare_read, "rope": _prepare_rope}[c["op"]](c, gen)


def _prepare_attention(c, gen):
    new, keys = _lengths(c)
    dt, bs, tokens = DTYPES[c["dtype"]], c["block_size"], sum(new)
    pages = [-(-k // bs) for k in keys]
    blocks = sum(pages) + 3
    order = torch.randperm(blocks, generator=gen, device="cuda")[: sum(pages)]
    first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
    column = torch.arange(max(pages), device="cuda")
    held = column[None] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.where(held, order[(first[:, None] + column).clamp(max=sum(pages) - 1)], -1)
    ckv, ckv_scale = _cache_part(gen, blocks * bs, DV, c["cache"], c["scale"])
    k, _ = _cache_part(gen, blocks * bs, DK, c["dtype"], "none")
    s = {"op": "attention", "block_size": bs, "longest": (max(new), max(keys)),
         "q_nope": torch.randn(tokens, c["heads"], DV, generator=gen, device="cuda").to(dt),
         "q_rope": torch.randn(tokens, c["heads"], DK, generator=gen, device="cuda").to(dt),
         "ckv": ckv.view(blocks, bs, 1, DV), "k": k.view(blocks, bs, 1, DK), "ckv_scale": ckv_scale, "table": table,
         "query_start": torch.tensor([0] + new, device="cuda").cumsum(0), "key_length": torch.tensor(keys, device="cuda"),
         "out": torch.empty(tokens, c["heads"], DV, device="cuda", dtype=dt),
         "lse": torch.empty(tokens, c["heads"], device="cuda") if c["lse"] else None}
    if own:   # the bound call that a serving loop keeps for its buffers
        import attention_prologue_kv_gb300 as kvr
        s["call"] = kvr.prepare_mla_attention(s["q_nope"], s["q_rope"], s["ckv"], s["k"], s["table"], s["query_start"],
                                              s["key_length"], s["out"], softmax_scale=SOFTMAX_SCALE, ckv_scale=ckv_scale,
                                              lse=s["lse"])
    return s


def _prepare_read(c, gen):
    n, tokens, bs, dt = c["seqs"], c["tokens"], c["block_size"], DTYPES[c["dtype"]]
    if c["mode"] == "Norm":
        blocks = n
        index = torch.rand(n, bs, generator=gen, device="cuda").argsort(1)[:, :tokens].reshape(-1)
    elif c["mode"] == "PA_BSND":
        blocks = -(-n * tokens // bs) * 2
        index = torch.randperm(blocks * bs, generator=gen, device="cuda")[: n * tokens]
    else:
        blocks = n * -(-tokens // bs) * 2
        index = torch.randperm(blocks, generator=gen, device="cuda")[: blocks // 2] * bs
    if c["skip"]:
        index[torch.randperm(index.numel(), generator=gen, device="cuda")[: c["skip"]]] = -1
    ckv, ckv_scale = _cache_part(gen, blocks * bs, DV, c["cache"], c["scale"])
    k, k_scale = _cache_part(gen, blocks * bs, DK, c["k_cache"] if c["k_cache"] not in ("bf16", "f16") else c["dtype"], c["scale"])
    s = {"op": "read", "mode": c["mode"], "ckv": ckv.view(blocks, bs, 1, DV), "k": k.view(blocks, bs, 1, DK),
         "ckv_scale": ckv_scale, "k_scale": k_scale, "index": index,
         "out": torch.zeros(n, 1, tokens, DV + DK, device="cuda", dtype=dt)}
    if own:
        import attention_prologue_kv_gb300 as kvr
        s["call"] = kvr.prepare_kv_cache_read(s["ckv"], s["k"], index, s["out"], cache_mode=c["mode"], ckv_scale=ckv_scale,
                                              k_scale=k_scale)
    return s


def _sections(pairs, axes):
    """Pairs of each axis: the first (time) has what is left over."""
    return [pairs - (axes - 1) * (pairs // axes)] + [pairs // axes] * (axes - 1)


def _prepare_rope(c, gen):
    t, dt = c["tokens"], DTYPES[c["dtype"]]
    q = torch.randn(t, c["heads"], c["wide"] + c["dim"], generator=gen, device="cuda").to(dt)[..., c["wide"]:]
    far = torch.tensor([131072] + [4096] * (c["axes"] - 1), device="cuda")[:, None]
    positions = (torch.rand(c["axes"], t, generator=gen, device="cuda", dtype=torch.float64) * far).to(torch.int64)
    table = lambda: torch.empty(t, c["dim"], device="cuda", dtype=dt) if c["tables"] else None  # noqa: E731
    s = {"op": "rope", "q": q, "positions": positions, "sections": _sections(c["dim"] // 2, c["axes"]),
         "layout": c["layout"], "out": torch.empty(t, c["heads"], c["dim"], device="cuda", dtype=dt), "cos": table(),
         "sin": table()}
    if own:
        import attention_prologue_kv_gb300 as kvr
        s["call"] = kvr.prepare_query_rope(q, positions, s["out"], sections=s["sections"], rope_layout=c["layout"],
                                           cos_out=s["cos"], sin_out=s["sin"])
    return s


def run(s):
    if own:
        s["call"]()
    else:
        {"attention": _plain_attention, "read": _plain_read, "rope": _plain_rope}[s["op"]](s)
    if s["op"] == "attention":
        return {"out": s["out"], "lse": s["lse"]} if s["lse"] is not None else {"out": s["out"]}
    if s["op"] == "read":
        return {"out": s["out"]}
    return {"out": s["out"], "cos": s["cos"], "sin": s["sin"]} if s["cos"] is not None else {"out": s["out"]}


def _dequantised(codes, scale):
    return codes.to(torch.float32) if scale is None else codes.to(torch.float32) / scale


def _plain_attention(s):
    """softmax(scale * (q_nope . c + q_rope . k)) c over the keys that token j of a sequence sees: those before
    key_length - new + j + 1."""
    longest_new, longest_keys = s["longest"]
    start, keys = s["query_start"], s["key_length"]
    heads = s["q_nope"].shape[1]
    new = start[1:] - start[:-1]
    step = torch.arange(longest_new, device="cuda")
    place = torch.arange(longest_keys, device="cuda")
    token = (start[:-1, None] + step).clamp(max=s["q_nope"].shape[0] - 1)
    q = torch.cat([s["q_nope"], s["q_rope"]], -1).to(torch.float32)[token].flatten(1, 2)
    page = s["table"][:, place // s["block_size"]].clamp(min=0)
    slot = page * s["block_size"] + place % s["block_size"]
    latent = _dequantised(s["ckv"].view(-1, DV)[slot], s["ckv_scale"])
    key = torch.cat([latent, s["k"].view(-1, DK)[slot].to(torch.float32)], -1)
    scores = (q @ key.transpose(1, 2)).mul_(SOFTMAX_SCALE).unflatten(1, (longest_new, heads))
    seen = place[None, None] < (keys - new)[:, None, None] + step[None, :, None] + 1
    scores = scores.masked_fill_(~seen[:, :, None], -torch.inf).flatten(1, 2)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, p @ latent / total, 0).unflatten(1, (longest_new, heads))
    row = torch.arange(s["q_nope"].shape[0], device="cuda")
    of = torch.searchsorted(start, row, right=True) - 1
    s["out"].copy_(out[of, row - start[of]])
    if s["lse"] is not None:
        s["lse"].copy_((top + total.log()).unflatten(1, (longest_new, heads))[of, row - start[of], :, 0])


def _rows_of_index(s):
    """Cache row of each output row, -1 where the index skips it."""
    index, bs = s["index"], s["ckv"].shape[1]
    n, tokens = s["out"].shape[0], s["out"].shape[2]
    if s["mode"] == "Norm":
        return torch.where(index < 0, -1, index + torch.arange(n, device="cuda").repeat_interleave(tokens) * bs)
    if s["mode"] == "PA_BSND":
        return index
    t = torch.arange(tokens, device="cuda")
    entry = index.view(n, -1)[:, t // bs]
    return torch.where(entry < 0, -1, entry + t % bs).reshape(-1)


def _plain_read(s):
    rows = _rows_of_index(s)
    at = rows.clamp(min=0)
    got = torch.cat([_dequantised(s["ckv"].view(-1, DV)[at], s["ckv_scale"]), _dequantised(s["k"].view(-1, DK)[at], s["k_scale"])], -1)
    flat = s["out"].view(-1, DV + DK)
    flat.copy_(torch.where(rows[:, None] < 0, flat, got.to(flat.dtype)))


def _plain_rope(s):
    """Pair i of a head turned by the position on its axis times 10000^(-2i / dim); angles in 64 bits."""
    dim = s["q"].shape[-1]
    half = dim // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    axis = torch.arange(len(s["sections"]), device="cuda").repeat_interleave(torch.tensor(s["sections"], device="cuda"), output_size=half)
    angle = s["positions"].to(torch.float64)[axis].T * 10000.0 ** (-2 * i / dim)
    cos, sin = angle.cos().to(torch.float32)[:, None], angle.sin().to(torch.float32)[:, None]
    q = s["q"].to(torch.float32)
    a, b = (q[..., 0::2], q[..., 1::2]) if s["layout"] == "interleave" else (q[..., :half], q[..., half:])
    s["out"].copy_(torch.cat([a * cos - b * sin, b * cos + a * sin], -1))
    if s["cos"] is not None:
        s["cos"].copy_(torch.cat([cos, cos], -1)[:, 0])
        s["sin"].copy_(torch.cat([sin, sin], -1)[:, 0])


def exact(c, seed):
    """The same from the definition, in 64 bits, sequence by sequence and a few rows at a time."""
    s = prepare(c, seed)
    wide = torch.float64
    if c["op"] == "attention":
        new, keys = _lengths(c)
        heads, bs, at = c["heads"], c["block_size"], 0
        out = torch.zeros(sum(new), heads, DV, device="cuda", dtype=wide)
        lse = torch.zeros(sum(new), heads, device="cuda", dtype=wide)
        for n, (count, length) in enumerate(zip(new, keys)):
            pages = s["table"][n, : -(-length // bs)]
            c_rows = s["ckv"][pages].reshape(-1, DV)[:length].to(wide)
            if s["ckv_scale"] is not None:
                c_rows = c_rows / s["ckv_scale"].to(wide)
            k_rows = s["k"][pages].reshape(-1, DK)[:length].to(wide)
            few = max(1, 400_000_000 // (heads * length))
            for j in range(0, count, few):
                m = min(few, count - j)
                qn, qr = s["q_nope"][at + j: at + j + m].to(wide), s["q_rope"][at + j: at + j + m].to(wide)
                x = SOFTMAX_SCALE * (torch.einsum("thd,kd->thk", qn, c_rows) + torch.einsum("thd,kd->thk", qr, k_rows))
                sees = length - count + j + torch.arange(m, device="cuda")   # the last key that each token sees
                x[torch.arange(length, device="cuda")[None, None].gt(sees[:, None, None]).expand_as(x)] = -torch.inf
                lse[at + j: at + j + m] = torch.logsumexp(x, -1)
                out[at + j: at + j + m] = torch.einsum("thk,kd->thd", torch.softmax(x, -1), c_rows)
                del x
            at += count
        return {"out": out, "lse": lse} if c["lse"] else {"out": out}
    if c["op"] == "read":
        n, tokens, bs = c["seqs"], c["tokens"], c["block_size"]
        out = s["out"].to(wide)
        index = s["index"].view(n, -1).tolist()
        parts = [(s["ckv"], s["ckv_scale"], slice(0, DV)), (s["k"], s["k_scale"], slice(DV, DV + DK))]
        for b in range(n):
            to, of = [], []
            for t in range(tokens):
                e = index[b][t // bs if c["mode"] == "PA_BLK_BSND" else t]
                if e >= 0:
                    to.append(t)
                    of.append(e + t % bs if c["mode"] == "PA_BLK_BSND" else e + b * bs if c["mode"] == "Norm" else e)
            for cache, scale, where in parts:
                rows = cache.reshape(-1, cache.shape[-1])[torch.tensor(of, device="cuda", dtype=torch.int64)].to(wide)
                out[b, 0, torch.tensor(to, device="cuda", dtype=torch.int64), where] = rows if scale is None else rows / scale.to(wide)
        return {"out": out}
    dim = c["dim"]
    half, q = dim // 2, s["q"].to(wide)
    out, cos, sin = torch.zeros_like(q), torch.zeros(c["tokens"], dim, device="cuda", dtype=wide), torch.zeros(c["tokens"], dim, device="cuda", dtype=wide)
    ends = [sum(s["sections"][: a + 1]) for a in range(c["axes"])]
    for i in range(half):
        turn = s["positions"][next(a for a, e in enumerate(ends) if i < e)].to(wide) * 10000.0 ** (-2.0 * i / dim)
        z = torch.polar(torch.ones_like(turn), turn)
        x, y = (2 * i, 2 * i + 1) if c["layout"] == "interleave" else (i, i + half)
        r = torch.complex(q[..., x], q[..., y]) * z[:, None]
        out[..., i], out[..., i + half] = r.real, r.imag
        cos[:, i] = cos[:, i + half] = z.real
        sin[:, i] = sin[:, i + half] = z.imag
    return {"out": out, "cos": cos, "sin": sin} if c["tables"] else {"out": out}
