"""What is measured of a latent cache of bounded size under drafted tokens: the ancestors of a tree of drafted tokens
(`draft_tree`), attention of such a tree over the cache (`mla_attention` with a tree mask), the attention weight that each
key receives (`mla_key_weight`), which keys to keep by it (`kv_cache_select`) and moving kept rows together
(`kv_cache_compact`), each in plain torch operations and as the library's call.

The head split is the one of the repository's workloads: Dv = 512 latent channels and Dk = 64 rotary channels, one key row
per token for all heads.
"""
import math
import random

import torch

own = False

DV, DK = 512, 64
SOFTMAX_SCALE = 0.0722   # scores of N(0, 1) queries and keys then spread over about +-5, as trained heads do
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.int8,
          "fp8_e4m3fn": torch.float8_e4m3fn, "fp8_e5m2": torch.float8_e5m2}


def listed():
    return [
        # the drafted tree of one conversation
        tree_case("tree_one", seqs=1, new=(26, 26), lengths=1),
        # those of a full batch, some of more than 64 tokens: two words a token
        tree_case("tree_batch", seqs=256, new=(9, 127), lengths=2),
        # that tree verified on one of eight cards that share the heads: latency
        attention_case("verify_one", seqs=1, new=(26, 26), keys=(1026, 1026), heads=16, lengths=3),
        # trees of a batch verified at once, every head on this card, contexts of all ages
        attention_case("verify_batch", seqs=48, new=(8, 31), keys=(500, 6000), heads=128, lengths=4),
        # weights of one conversation's keys after a step
        weight_case("weight_one", seqs=1, new=(1, 1), keys=(1000, 1000), heads=16, lengths=5, dtype="f16"),
        # the same of a full decode batch
        weight_case("weight_batch", seqs=256, new=(1, 1), keys=(1, 4095), heads=128, lengths=6),
        # the last tokens of prompts, whose weights decide what of the prompt stays, over an 8-bit cache
        weight_case("weight_window_fp8", seqs=8, new=(17, 32), keys=(3000, 8192), heads=128, cache="fp8_e4m3fn",
                    scale="channel", decay=0.0, lengths=7),
        # every query of a long chunk: the largest
        weight_case("weight_chunk", seqs=1, new=(512, 512), keys=(16384, 16384), heads=128, lengths=8),
        # one long conversation cut to a quarter
        select_case("select_long", seqs=1, keys=(131000, 131000), keep=32768, sink=4, recent=512, lengths=9),
        # a batch at its limit
        select_case("select_batch", seqs=64, keys=(2048, 4095), keep=2048, sink=4, recent=128, lengths=10),
        # the accepted branch of each tree moved behind its context
        compact_case("compact_accepted", seqs=256, keys=(200, 4000), new=(9, 31), keep=(1, 7), lengths=11),
        # the kept half of each sequence moved to its front
        compact_case("compact_evicted", seqs=64, keys=(4000, 4096), new=(0, 0), keep=(2000, 2048), lengths=12),
    ]


def _named(name, c):
    return dict(c, name=name) if name else c


def tree_case(name, seqs, new, lengths):
    return _named(name, {"op": "tree", "seqs": seqs, "new_min": new[0], "new_max": new[1], "lengths": lengths})


def attention_case(name, seqs, new, keys, heads, lengths, dtype="bf16", cache="bf16", scale="none", block_size=128, lse=True):
    return _named(name, {"op": "attention", "seqs": seqs, "new_min": new[0], "new_max": new[1], "keys_min": keys[0],
                         "keys_max": keys[1], "heads": heads, "lengths": lengths, "dtype": dtype,
                         "cache": dtype if cache == "bf16" else cache, "scale": scale, "block_size": block_size, "lse": lse})


def weight_case(name, seqs, new, keys, heads, lengths, dtype="bf16", cache="bf16", scale="none", block_size=128, decay=1.0):
    """decay 0: no weights of earlier steps are taken up."""
    return _named(name, {"op": "weight", "seqs": seqs, "new_min": new[0], "new_max": new[1], "keys_min": keys[0],
                         "keys_max": keys[1], "heads": heads, "lengths": lengths, "dtype": dtype,
                         "cache": dtype if cache == "bf16" else cache, "scale": scale, "block_size": block_size, "decay": decay})


def select_case(name, seqs, keys, keep, sink, recent, lengths):
    return _named(name, {"op": "select", "seqs": seqs, "keys_min": keys[0], "keys_max": keys[1], "new_min": 1, "new_max": 1,
                         "keep": keep, "sink": sink, "recent": recent, "lengths": lengths})


def compact_case(name, seqs, keys, new, keep, lengths, dtype="bf16", cache="bf16", block_size=128):
    """new > 0: `keep` of the last `new` keys move to the front of these; new = 0: `keep` of all keys to the very front."""
    return _named(name, {"op": "compact", "seqs": seqs, "keys_min": keys[0], "keys_max": keys[1], "new_min": new[0],
                         "new_max": new[1], "keep_min": keep[0], "keep_max": keep[1], "lengths": lengths, "dtype": dtype,
                         "cache": dtype if cache == "bf16" else cache, "block_size": block_size})


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["tree", "attention", "attention", "weight", "weight", "weight", "select", "compact"])
    lengths = rng.randint(1, 10 ** 6)
    if op == "tree":
        most = _log_int(rng, 1, 200)
        return tree_case(None, _log_int(rng, 1, 512), (rng.randint(1, most), most), lengths)
    if op == "select":
        keys = _log_int(rng, 2, 131072)
        keep = rng.randint(1, keys)
        sink = rng.randint(0, min(8, keep))
        return select_case(None, max(1, min(_log_int(rng, 1, 256), 4000000 // keys)), (rng.randint(1, keys), keys), keep, sink,
                           rng.randint(0, min(1000, keep - sink)), lengths)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([dtype, dtype, "int8", "fp8_e4m3fn", "fp8_e5m2"])
    scale = "none" if cache == dtype else rng.choice(["channel", "tensor"])
    block = rng.choice([16, 32, 64, 100, 128, 256])
    if op == "compact":
        keys = _log_int(rng, 8, 32768)
        seqs = max(1, min(_log_int(rng, 1, 256), 300000 // keys))
        if rng.random() < 0.5:
            new = rng.randint(1, min(keys, 64))
            return compact_case(None, seqs, (new, keys), (new, new), (1, rng.randint(1, new)), lengths, dtype, cache, block)
        keep = rng.randint(1, keys // 2)
        return compact_case(None, seqs, (keys - keys // 8, keys), (0, 0), (max(1, keep // 2), keep), lengths, dtype, cache, block)
    heads = _log_int(rng, 1, 128)
    most_new = _log_int(rng, 1, 200 if op == "attention" else 512)
    most_keys = _log_int(rng, max(8, most_new), 16384)
    # at most about the rows x keys of the largest listed case of the operator, and as many keys as the largest decode batch
    cells = 300000000 if op == "attention" else 500000000
    seqs = max(1, min(_log_int(rng, 1, 256), cells // (most_new * heads * most_keys), 600000 // most_keys))
    new, keys = (rng.randint(1, most_new), most_new), (rng.randint(1, most_keys), most_keys)
    if op == "attention":
        return attention_case(None, seqs, new, keys, heads, lengths, dtype, cache, scale, block, scale != "channel")
    return weight_case(None, seqs, new, keys, heads, lengths, dtype, cache, scale, block, rng.choice([0.0, 0.5, 1.0]))


def _lengths(c):
    """New tokens and keys (the new ones among them) of each sequence; the case's own, whatever the seed."""
    r = random.Random(c["lengths"])
    new = [r.randint(c["new_min"], c["new_max"]) for _ in range(c["seqs"])]
    keys = [max(n, r.randint(c["keys_min"], c["keys_max"])) for n in new] if "keys_min" in c else new
    return new, keys


def _kept_counts(c):
    """Rows that compact keeps of each sequence."""
    new, keys = _lengths(c)
    r = random.Random(c["lengths"] + 1)
    return [min(r.randint(c["keep_min"], c["keep_max"]), n if c["new_max"] else k) for n, k in zip(new, keys)]


def _row_bytes(c):
    return DV * (2 if c["cache"] in ("bf16", "f16") else 1) + DK * 2


def work(c):
    new, keys = _lengths(c)
    if c["op"] == "tree":
        words = -(-max(new) // 64)
        return {"bytes": sum(new) * (16 + 8 * words) + 16 * len(new) + 8, "flops": sum(new) * math.log(1 + max(new))}
    if c["op"] == "select":
        kept = sum(min(k, c["keep"]) for k in keys)
        return {"bytes": 4 * sum(keys) + 8 * len(keys) * (c["keep"] + 2) + 4 * kept, "flops": sum(keys)}
    if c["op"] == "compact":
        kept = _kept_counts(c)
        moved = sum(max(0, m - 1) for m in kept)   # the first one stays
        return {"bytes": 2 * moved * _row_bytes(c) + 8 * (sum(kept) + 2 * len(kept)), "flops": moved}
    rows = sum(new) * c["heads"]
    pages = sum(-(-k // c["block_size"]) for k in keys)
    shared = rows * (DV + DK) * 2 + sum(keys) * _row_bytes(c) + 8 * (pages + 2 * len(keys) + 1)
    shared += {"none": 0, "tensor": 4, "channel": 4 * DV}[c["scale"]]
    if c["op"] == "attention":
        # keys before the tree, and a token's ancestors: of token j about 1 + 1 + 1/2 + ... + 1/j
        pairs = sum(n * (k - n) + sum(1 + math.log(1 + j) for j in range(n)) for n, k in zip(new, keys))
        words = -(-max(new) // 64)
        return {"bytes": shared + rows * DV * 2 + sum(new) * 8 * words + (4 * rows if c["lse"] else 0),
                "flops": 2 * pairs * c["heads"] * (DV + DK + DV)}
    pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(new, keys))
    return {"bytes": shared + 4 * rows + sum(keys) * (8 if c["decay"] else 4), "flops": 2 * pairs * c["heads"] * (DV + DK)}


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"tree": _prepare_tree, "attention": _prepare_attention, "weight": _prepare_weight, "select": _prepare_select,
         "compact": _prepare_compact}[c["op"]](c, gen)
    if own:   # the bound call that a serving loop keeps for its buffers
        s["call"] = _bind(s)
    return s


def _bind(s):
    import attention_prologue_kv_gb300 as kvr
    if s["op"] == "tree":
        return kvr.prepare_draft_tree(s["parent"], s["query_start"], s["mask"], position_start=s["position_start"],
                                      positions=s["positions"])
    if s["op"] == "attention":
        return kvr.prepare_mla_attention(s["q_nope"], s["q_rope"], s["ckv"], s["k"], s["table"], s["query_start"],
                                         s["key_length"], s["out"], softmax_scale=SOFTMAX_SCALE, ckv_scale=s["ckv_scale"],
                                         lse=s["lse"], tree_mask=s["mask"])
    if s["op"] == "weight":
        return kvr.prepare_mla_key_weight(s["q_nope"], s["q_rope"], s["ckv"], s["k"], s["table"], s["query_start"],
                                          s["key_length"], s["lse"], s["weight"], softmax_scale=SOFTMAX_SCALE,
                                          ckv_scale=s["ckv_scale"], past=s["past"], decay=s["decay"])
    if s["op"] == "select":
        return kvr.prepare_kv_cache_select(s["weight"], s["key_length"], s["kept"], s["kept_length"], sink=s["sink"],
                                           recent=s["recent"], kept_weight=s["kept_weight"])
    return kvr.prepare_kv_cache_compact(s["ckv"], s["k"], s["table"], s["kept"], s["kept_length"], start=s["start"])


def _starts(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0)


def _parents(counts, gen):
    """Each first token follows the context, every other one a token before it: [T], places in the sequence."""
    start = _starts(counts)
    place = torch.arange(int(sum(counts)), device="cuda") - start[:-1].repeat_interleave(torch.tensor(counts, device="cuda"))
    u = torch.rand(place.shape[0], generator=gen, device="cuda", dtype=torch.float64)
    return torch.where(place == 0, -1, (u * place).long())


def _prepare_tree(c, gen):
    new, _ = _lengths(c)
    total, words = sum(new), -(-max(new) // 64)
    begin = (torch.rand(len(new), generator=gen, device="cuda", dtype=torch.float64) * 131072).long()
    return {"op": "tree", "longest": max(new), "parent": _parents(new, gen), "query_start": _starts(new), "position_start": begin,
            "mask": torch.zeros(total, words, dtype=torch.int64, device="cuda"),
            "positions": torch.zeros(total, dtype=torch.int64, device="cuda")}


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


def _pages(keys, bs, gen):
    """(block table [N, most pages], blocks): the sequences' pages in no order, -1 behind their last."""
    pages = [-(-k // bs) for k in keys]
    blocks = sum(pages) + 3
    order = torch.randperm(blocks, generator=gen, device="cuda")[: sum(pages)]
    column = torch.arange(max(pages), device="cuda")
    held = column[None] < torch.tensor(pages, device="cuda")[:, None]
    return torch.where(held, order[(_starts(pages)[:-1, None] + column).clamp(max=sum(pages) - 1)], -1), blocks


def _prepare_step(c, gen):
    """Queries, caches and lengths, as attention and weights share them."""
    new, keys = _lengths(c)
    dt, bs, tokens = DTYPES[c["dtype"]], c["block_size"], sum(new)
    table, blocks = _pages(keys, bs, gen)
    ckv, ckv_scale = _cache_part(gen, blocks * bs, DV, c["cache"], c["scale"])
    k, _ = _cache_part(gen, blocks * bs, DK, c["dtype"], "none")
    return {"op": c["op"], "block_size": bs, "longest": (max(new), max(keys)),
            "q_nope": torch.randn(tokens, c["heads"], DV, generator=gen, device="cuda").to(dt),
            "q_rope": torch.randn(tokens, c["heads"], DK, generator=gen, device="cuda").to(dt),
            "ckv": ckv.view(blocks, bs, 1, DV), "k": k.view(blocks, bs, 1, DK), "ckv_scale": ckv_scale, "table": table,
            "query_start": _starts(new), "key_length": torch.tensor(keys, device="cuda")}


def _prepare_attention(c, gen):
    s = _prepare_step(c, gen)
    new, _ = _lengths(c)
    s["mask"] = _ancestor_words(_parents(new, gen), s["query_start"], max(new))[0]
    s["out"] = torch.empty_like(s["q_nope"])
    s["lse"] = torch.empty(s["q_nope"].shape[:2], device="cuda") if c["lse"] else None
    return s


def _prepare_weight(c, gen):
    s = _prepare_step(c, gen)
    _, _, scores = _plain_scores(s)   # [N, new, H, keys], -inf where a token does not see a key
    lse = torch.logsumexp(scores, -1)
    row = torch.arange(s["q_nope"].shape[0], device="cuda")
    of = torch.searchsorted(s["query_start"], row, right=True) - 1
    s["lse"] = lse[of, row - s["query_start"][of]].contiguous()
    n, width = len(s["key_length"]), s["table"].shape[1] * s["block_size"]
    s["decay"] = c["decay"]
    s["past"] = torch.rand(n, width, generator=gen, device="cuda") * c["heads"] if c["decay"] else None
    s["weight"] = torch.zeros(n, width, device="cuda")
    return s


def _prepare_select(c, gen):
    _, keys = _lengths(c)
    n, width = c["seqs"], max(keys)
    # a few keys of large weight, most of little, some of none
    weight = (torch.randn(n, width, generator=gen, device="cuda") * 2).exp()
    weight = torch.where(torch.rand(n, width, generator=gen, device="cuda") < 0.1, 0.0, weight)
    return {"op": "select", "weight": weight, "key_length": torch.tensor(keys, device="cuda"), "sink": c["sink"], "recent": c["recent"],
            "kept": torch.zeros(n, c["keep"], dtype=torch.int64, device="cuda"),
            "kept_length": torch.zeros(n, dtype=torch.int64, device="cuda"),
            "kept_weight": torch.zeros(n, c["keep"], device="cuda")}


def _prepare_compact(c, gen):
    """The first of a sequence's rows stays, the others come from behind the place that they go to."""
    new, keys = _lengths(c)
    count = _kept_counts(c)
    bs, n, most = c["block_size"], c["seqs"], max(count)
    table, blocks = _pages(keys, bs, gen)
    span = torch.tensor([a if c["new_max"] else b for a, b in zip(new, keys)], device="cuda")
    m = torch.tensor(count, device="cuda")
    # m - 1 places of [m, span), ascending; where there are fewer, the row stays
    place = torch.arange(most, device="cuda")
    room = (span - m)[:, None]
    u = torch.rand(n, most, generator=gen, device="cuda", dtype=torch.float64).sort(1).values
    step = torch.minimum((u * (room - m[:, None] + 2).clamp(min=0)).long(), (room - m[:, None] + 1).clamp(min=0))
    kept = torch.where((place[None] > 0) & (room >= m[:, None] - 1), m[:, None] + place - 1 + step.sort(1).values, place[None])
    start = torch.tensor([b - a if c["new_max"] else 0 for a, b in zip(new, keys)], device="cuda")
    ckv, _ = _cache_part(gen, blocks * bs, DV, c["cache"], "tensor")
    k, _ = _cache_part(gen, blocks * bs, DK, c["dtype"], "none")
    return {"op": "compact", "block_size": bs, "ckv": ckv.view(blocks, bs, 1, DV), "k": k.view(blocks, bs, 1, DK), "table": table,
            "kept": (torch.where(place[None] < m[:, None], kept + start[:, None], -1)).contiguous(), "kept_length": m, "start": start}


def run(s):
    if own:
        s["call"]()
    else:
        {"tree": _plain_tree, "attention": _plain_attention, "weight": _plain_weight, "select": _plain_select,
         "compact": _plain_compact}[s["op"]](s)
    if s["op"] == "tree":
        return {"mask": s["mask"], "positions": s["positions"]}
    if s["op"] == "attention":
        return {"out": s["out"], "lse": s["lse"]} if s["lse"] is not None else {"out": s["out"]}
    if s["op"] == "weight":
        return {"weight": s["weight"]}
    if s["op"] == "select":
        return {"kept": s["kept"], "kept_length": s["kept_length"], "kept_weight": s["kept_weight"]}
    return {"ckv": s["ckv"], "k": s["k"]}


def _ancestor_words(parent, start, longest):
    """(words [T, longest / 64], depth [T]): the ancestors of a token, itself among them. With P[j, parent of j] = 1 they
    are the ones of (1 - P)^-1 = 1 + P + P^2 + ..."""
    row = torch.arange(parent.shape[0], device="cuda")
    of = torch.searchsorted(start, row, right=True) - 1
    place = row - start[of]
    step = torch.zeros(start.shape[0] - 1, longest, longest + 1, device="cuda")
    step[of, place, torch.where(parent < 0, longest, parent)] = 1
    one = torch.eye(longest, device="cuda")
    ancestors = torch.linalg.solve_triangular(one - step[:, :, :longest], one.expand(start.shape[0] - 1, longest, longest), upper=False)
    mine = torch.nn.functional.pad(ancestors[of, place].long(), (0, -longest % 64))
    return (mine.unflatten(1, (-1, 64)) << torch.arange(64, device="cuda")).sum(-1), mine.sum(-1) - 1


def _plain_tree(s):
    words, depth = _ancestor_words(s["parent"], s["query_start"], s["longest"])
    s["mask"].copy_(words)
    row = torch.arange(words.shape[0], device="cuda")
    s["positions"].copy_(s["position_start"][torch.searchsorted(s["query_start"], row, right=True) - 1] + depth)


def _plain_scores(s):
    """(latent rows, whether a token sees a key, scaled scores [N, new, H, keys] with -inf where it does not): a token sees
    the keys before its sequence's new ones, and of these its ancestors, or with no tree those up to itself."""
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
    latent = s["ckv"].view(-1, DV)[slot].to(torch.float32)
    if s["ckv_scale"] is not None:
        latent = latent / s["ckv_scale"]
    key = torch.cat([latent, s["k"].view(-1, DK)[slot].to(torch.float32)], -1)
    scores = (q @ key.transpose(1, 2)).mul_(SOFTMAX_SCALE).unflatten(1, (longest_new, heads))
    before = (keys - new)[:, None]
    if "mask" in s:
        bit = place[None] - before   # place among the new tokens
        word = s["mask"][token].gather(2, (bit >> 6).clamp(0, s["mask"].shape[1] - 1)[:, None].expand(-1, longest_new, -1))
        seen = (bit < 0)[:, None] | (((word >> (bit & 63)[:, None]) & 1) == 1) & (bit < new[:, None])[:, None]
    else:
        seen = place[None, None] < before[:, :, None] + step[None, :, None] + 1
    seen = seen & (step[None] < new[:, None])[:, :, None]
    return latent, seen, scores.masked_fill_(~seen[:, :, None], -torch.inf)


def _plain_attention(s):
    """softmax(scale * (q_nope . c + q_rope . k)) c over the keys that a token sees."""
    latent, _, scores = _plain_scores(s)
    longest_new, heads = scores.shape[1:3]
    scores = scores.flatten(1, 2)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, p @ latent / total, 0).unflatten(1, (longest_new, heads))
    row = torch.arange(s["q_nope"].shape[0], device="cuda")
    of = torch.searchsorted(s["query_start"], row, right=True) - 1
    s["out"].copy_(out[of, row - s["query_start"][of]])
    if s["lse"] is not None:
        s["lse"].copy_((top + total.log()).unflatten(1, (longest_new, heads))[of, row - s["query_start"][of], :, 0])


def _plain_weight(s):
    """decay * past + the sum of exp(score - lse) over the tokens and heads of a sequence, for each of its keys."""
    _, seen, scores = _plain_scores(s)
    token = (s["query_start"][:-1, None] + torch.arange(scores.shape[1], device="cuda")).clamp(max=s["lse"].shape[0] - 1)
    total = scores.sub_(s["lse"][token][..., None]).exp_().sum((1, 2))
    mine = s["weight"][:, : total.shape[1]]
    held = torch.arange(total.shape[1], device="cuda")[None] < s["key_length"][:, None]
    if s["past"] is not None:
        total = total + s["decay"] * s["past"][:, : total.shape[1]]
    mine.copy_(torch.where(held, total, mine))


def _plain_select(s):
    """The first `sink` keys, the last `recent` ones and of the others those of largest weight, the earlier of equal ones."""
    place = torch.arange(s["weight"].shape[1], device="cuda")[None]
    keys = s["key_length"][:, None]
    keep = s["kept"].shape[1]
    rank = torch.where((place < s["sink"]) | (place >= keys - s["recent"]), torch.inf, s["weight"])
    rank = torch.where(place < keys, rank, -torch.inf)
    first = rank.sort(dim=1, descending=True, stable=True).indices[:, :keep]
    count = keys.clamp(max=keep)
    behind = torch.arange(keep, device="cuda")[None] >= count
    first = torch.nn.functional.pad(first, (0, keep - first.shape[1]))
    kept = torch.where(behind, place.shape[1], first).sort(1).values
    s["kept"].copy_(torch.where(behind, -1, kept))
    s["kept_length"].copy_(count[:, 0])
    s["kept_weight"].copy_(torch.where(behind, 0, s["weight"].gather(1, kept.clamp(max=place.shape[1] - 1))))


def _plain_compact(s):
    """Rows read first, then written at start, start + 1, ..."""
    place = torch.arange(s["kept"].shape[1], device="cuda")[None]
    held = place < s["kept_length"][:, None]
    of, to = s["kept"].clamp(min=0), s["start"][:, None] + place
    bs, last = s["block_size"], s["table"].shape[1] - 1
    slot = lambda x: s["table"].gather(1, (x // bs).clamp(max=last)) * bs + x % bs  # noqa: E731
    of, to = slot(of)[held], slot(to)[held]
    for_bytes = lambda x: x.view(-1, x.shape[-1]).view(torch.int8 if x.element_size() == 1 else torch.int16)  # noqa: E731
    ckv, k = for_bytes(s["ckv"]), for_bytes(s["k"])
    ckv[to], k[to] = ckv[of], k[of]


def _seen_by(c, s, n, j, count, length):
    """Places of the keys that token j of sequence n sees, from the parents' words."""
    if "mask" not in s:
        return length - count + j + 1, []
    words = s["mask"][int(s["query_start"][n]) + j].tolist()
    return length - count, [length - count + b for b in range(count) if words[b // 64] >> (b % 64) & 1]


def exact(c, seed):
    """The same from the definition, in 64 bits, sequence by sequence and a few rows at a time."""
    s = prepare(c, seed)
    wide = torch.float64
    new, keys = _lengths(c)
    if c["op"] == "tree":
        parent, at = s["parent"].tolist(), 0
        mask, positions = torch.zeros_like(s["mask"], device="cpu"), torch.zeros_like(s["positions"], device="cpu")
        for n, count in enumerate(new):
            lines = []
            for j in range(count):
                up = parent[at + j]
                lines.append((lines[up] if up >= 0 else set()) | {j})
                positions[at + j] = int(s["position_start"][n]) + len(lines[j]) - 1
                for b in lines[j]:
                    mask[at + j, b // 64] |= torch.tensor(1 << (b % 64) if b % 64 < 63 else -(1 << 63))
            at += count
        return {"mask": mask.cuda(), "positions": positions.cuda()}
    if c["op"] == "select":
        kept, count = torch.full_like(s["kept"], -1), torch.zeros_like(s["kept_length"])
        carried = torch.zeros_like(s["kept_weight"])
        for n, length in enumerate(keys):
            w = s["weight"][n, :length].tolist()
            sure = [i for i in range(length) if i < c["sink"] or i >= length - c["recent"]]
            order = sorted((i for i in range(c["sink"], length - c["recent"])), key=lambda i: (-w[i], i))
            mine = sorted((sure + order)[: c["keep"]]) if length > c["keep"] else list(range(length))
            kept[n, : len(mine)] = torch.tensor(mine, device="cuda")
            carried[n, : len(mine)] = s["weight"][n, torch.tensor(mine, device="cuda")]
            count[n] = len(mine)
        return {"kept": kept, "kept_length": count, "kept_weight": carried}
    if c["op"] == "compact":
        ckv, k = s["ckv"].clone(), s["k"].clone()
        raw = lambda x: x.view(-1, x.shape[-1]).view(torch.int8 if x.element_size() == 1 else torch.int16)  # noqa: E731
        bs, table = s["block_size"], s["table"].tolist()
        for n, count in enumerate(s["kept_length"].tolist()):
            start = int(s["start"][n])
            row = lambda x: table[n][x // bs] * bs + x % bs  # noqa: E731,B023
            of = torch.tensor([row(x) for x in s["kept"][n, :count].tolist()], device="cuda")
            to = torch.tensor([row(start + i) for i in range(count)], device="cuda")
            raw(ckv)[to] = raw(s["ckv"])[of]
            raw(k)[to] = raw(s["k"])[of]
        return {"ckv": ckv, "k": k}
    heads, bs, at = c["heads"], c["block_size"], 0
    weight = s["weight"].to(wide) if c["op"] == "weight" else None
    out = torch.zeros(sum(new), heads, DV, device="cuda", dtype=wide)
    lse = torch.zeros(sum(new), heads, device="cuda", dtype=wide)
    for n, (count, length) in enumerate(zip(new, keys)):
        pages = s["table"][n, : -(-length // bs)]
        c_rows = s["ckv"][pages].reshape(-1, DV)[:length].to(wide)
        if s["ckv_scale"] is not None:
            c_rows = c_rows / s["ckv_scale"].to(wide)
        k_rows = s["k"][pages].reshape(-1, DK)[:length].to(wide)
        few = max(1, 400_000_000 // (heads * length))
        if weight is not None:
            weight[n, :length] = s["decay"] * s["past"][n, :length].to(wide) if s["past"] is not None else 0
        for j in range(0, count, few):
            m = min(few, count - j)
            qn, qr = s["q_nope"][at + j: at + j + m].to(wide), s["q_rope"][at + j: at + j + m].to(wide)
            x = SOFTMAX_SCALE * (torch.einsum("thd,kd->thk", qn, c_rows) + torch.einsum("thd,kd->thk", qr, k_rows))
            hidden = torch.ones(m, length, dtype=torch.bool, device="cuda")
            for i in range(m):
                before, more = _seen_by(c, s, n, j + i, count, length)
                hidden[i, :before] = False
                if more:
                    hidden[i, torch.tensor(more, device="cuda")] = False
            x.masked_fill_(hidden[:, None], -torch.inf)
            if weight is not None:
                weight[n, :length] += torch.exp(x - s["lse"][at + j: at + j + m, :, None].to(wide)).sum((0, 1))
            else:
                lse[at + j: at + j + m] = torch.logsumexp(x, -1)
                out[at + j: at + j + m] = torch.einsum("thk,kd->thd", torch.softmax(x, -1), c_rows)
            del x
        at += count
    if weight is not None:
        return {"weight": weight}
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
