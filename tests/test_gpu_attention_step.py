"""The operators of an attention step together, as a model's step calls them,
and the ways of calling them: streams, graphs, bound calls, workspaces."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
from attention_helpers import SENTINEL, check_mla, mla_case, oracle_mla, run_mla
from attention_prologue_kv_gb300 import _native as N

pytestmark = pytest.mark.gpu

H, DV, DK, BS = 16, 512, 64, 32
SCALE = 0.0722


def step_tensors(new, keys, seed):
    """A step's inputs: the new tokens' projections and positions, a cache that holds the earlier keys."""
    g = torch.Generator().manual_seed(seed)
    T, n = sum(new), len(new)
    pages = [-(-k // BS) for k in keys]
    blocks = sum(pages) + 1
    order = torch.randperm(blocks, generator=g)
    table = torch.full((n, max(pages)), -1, dtype=torch.int64)
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = order[at:at + p]
        at += p
    place = torch.cat([torch.arange(k - m, k) for m, k in zip(new, keys)])
    of = torch.repeat_interleave(torch.arange(n), torch.tensor(new))
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    d = dict(kv=bf(T, DV + DK), gamma=(torch.rand(DV, generator=g) + 0.5).to(torch.bfloat16), q_nope=bf(T, H, DV), q_pe=bf(T, H, DK),
             positions=torch.stack([place, place % 37, place % 11]), index=table[of, place // BS] * BS + place % BS, table=table,
             query_start=torch.tensor([0] + list(np.cumsum(new))), key_length=torch.tensor(keys),
             ckv=bf(blocks, BS, 1, DV), k=bf(blocks, BS, 1, DK))
    return {k: v.cuda() for k, v in d.items()}


def buffers(T):
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    return dict(q_rope=z(T, H, DK), cos=z(T, DK), sin=z(T, DK), out=z(T, H, DV), lse=torch.zeros(T, H, device="cuda"), back=z(T, DV + DK))


def one_step(s, b, **kw):
    """The key of the new tokens into the cache, their queries turned, attention over it, the new rows read back."""
    sections = [16, 8, 8]
    kvr.query_rope(s["q_pe"], s["positions"], b["q_rope"], sections=sections, cos_out=b["cos"], sin_out=b["sin"], **kw)
    kvr.kv_rmsnorm_rope_cache(s["kv"], s["gamma"], b["cos"], b["sin"], s["index"], s["ckv"], s["k"], **kw)
    kvr.mla_attention(s["q_nope"], b["q_rope"], s["ckv"], s["k"], s["table"], s["query_start"], s["key_length"], b["out"],
                      softmax_scale=SCALE, lse=b["lse"], **kw)
    kvr.kv_cache_read(s["ckv"], s["k"], s["index"], b["back"], **kw)


def expected_step(s):
    """The same in float64 torch, each intermediate rounded where the operators round it."""
    pos, f = s["positions"].double(), lambda t: t.double()  # noqa: E731
    axis = torch.repeat_interleave(torch.arange(3), torch.tensor([16, 8, 8])).cuda()
    ang = pos[axis].T * 10000.0 ** (-2 * torch.arange(32, device="cuda").double() / 64)
    cos, sin = torch.cat([ang.cos()] * 2, -1).bfloat16(), torch.cat([ang.sin()] * 2, -1).bfloat16()
    x = f(s["q_pe"])
    c, sn = ang.cos()[:, None], ang.sin()[:, None]
    q_rope = torch.cat([x[..., ::2] * c - x[..., 1::2] * sn, x[..., 1::2] * c + x[..., ::2] * sn], -1).bfloat16()
    left, right = f(s["kv"][:, :DV]), f(s["kv"][:, DV:])
    y = left / (left.square().mean(-1, keepdim=True) + float(np.float32(1e-6))).sqrt() * f(s["gamma"])
    x1, x2 = right[:, ::2], right[:, 1::2]
    rope = torch.cat([x1, x2], -1) * f(cos) + torch.cat([-x2, x1], -1) * f(sin)
    rows = torch.cat([y, rope], -1).bfloat16()
    ckv, k = s["ckv"].clone(), s["k"].clone()
    ckv.view(-1, DV)[s["index"]] = rows[:, :DV]
    k.view(-1, DK)[s["index"]] = rows[:, DV:]
    out = torch.zeros(s["q_nope"].shape, device="cuda", dtype=torch.float64)
    start, keys = s["query_start"].tolist(), s["key_length"].tolist()
    for n in range(len(keys)):
        i = torch.arange(keys[n], device="cuda")
        slot = s["table"][n, i // BS] * BS + i % BS
        cv, kr = f(ckv.view(-1, DV)[slot]), f(k.view(-1, DK)[slot])
        a, b = start[n], start[n + 1]
        sc = SCALE * (f(s["q_nope"][a:b]) @ cv.T + f(q_rope[a:b]) @ kr.T)
        sees = keys[n] - (b - a) + torch.arange(b - a, device="cuda") + 1
        sc = sc.masked_fill(i[None, None] >= sees[:, None, None], -torch.inf)
        out[a:b] = torch.softmax(sc, -1) @ cv
    return out, rows


def near(got, want, rel):
    return float((got.double() - want).norm() / want.norm()) <= rel


# Each intermediate may round to its other neighbour (a step of 2^-8 of a value, seldom), weights and the output by half
# a step (2^-9 on average of random signs well below that): 2^-7 in the 2-norm leaves them room, a wrong operator none.
STEP_REL = 2.0 ** -7


@pytest.mark.parametrize("new,keys", [([1] * 5, [1, 31, 200, 64, 33]), ([4, 1, 7], [4, 90, 300]), ([150], [420])])
def test_a_step(new, keys):
    s = step_tensors(new, keys, 1)
    b = buffers(sum(new))
    want, rows = expected_step(s)
    one_step(s, b)
    torch.cuda.synchronize()
    assert near(b["out"], want, STEP_REL)
    assert near(b["back"], rows.double(), 2.0 ** -9)
    assert torch.isfinite(b["lse"]).all()


def test_captured_and_replayed_on_new_inputs():
    """A step captured once; replays follow what the buffers hold: queries, caches, tables and lengths."""
    new, keys = [2, 1, 3], [70, 33, 130]
    s = step_tensors(new, keys, 2)
    b = buffers(6)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one_step(s, b)   # the first call on a device may not be captured (it looks up the kernels' limits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_step(s, b)
    for seed, lengths in ((3, [70, 33, 130]), (4, [65, 2, 99])):
        t = step_tensors(new, lengths, seed)
        for k in s:
            if k == "table":
                s[k].fill_(-1)
                s[k][:, :t[k].shape[1]] = t[k]
            elif k in ("ckv", "k"):
                n = min(s[k].shape[0], t[k].shape[0])
                s[k][:n] = t[k][:n]
                s[k][n:] = 0
            else:
                s[k].copy_(t[k])
        if int(s["table"].max()) >= s["ckv"].shape[0]:
            s["table"].clamp_(max=s["ckv"].shape[0] - 1)
        want, _ = expected_step(s)
        b["out"].fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert near(b["out"], want, STEP_REL)


def test_two_graphs_with_workspaces_of_their_own():
    """Two captured calls replayed at the same time on two streams give what they give alone."""
    cases = [mla_case([3, 1], [900, 1500], 24, block_size=64, seed=20), mla_case([1] * 30, [200] * 30, 16, cache="int8", scale_len=0, seed=21)]
    alone = [run_mla(c) for c in cases]
    graphs = []
    for c in cases:
        d = lambda t: None if t is None else t.cuda()  # noqa: E731
        args = [t.cuda().contiguous() for t in (c.q_nope, c.q_rope)] + [d(c.ckv), d(c.k), d(c.table), d(c.query_start), d(c.key_length)]
        out = torch.zeros(c.q_nope.shape, device="cuda", dtype=c.q_nope.dtype)
        call = kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale, ckv_scale=d(c.ckv_scale), k_scale=d(c.k_scale))
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, out, call))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for (g, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, out, _), ref in zip(graphs, alone):
        assert np.array_equal(out.double().cpu().numpy(), ref[0])


def test_streams():
    """On another stream than the current one, given or current: ordered after what that stream holds."""
    c = mla_case([2, 1], [300, 90], 8, block_size=32, seed=22)
    ref = run_mla(c)
    st = torch.cuda.Stream()
    got = run_mla(c, stream=st)
    assert np.array_equal(got[0], ref[0])
    got = run_mla(c, stream=st.cuda_stream)
    assert np.array_equal(got[0], ref[0])
    with torch.cuda.stream(st):
        got = run_mla(c)
    assert np.array_equal(got[0], ref[0])


def test_own_workspace_outlives_a_call_on_another_stream():
    """A bound call's own workspace goes to nobody else while a call of it waits or runs on another stream."""
    c = mla_case([2, 1], [300, 90], 8, block_size=32, seed=22)
    ref = run_mla(c)
    args = [t.cuda().contiguous() for t in (c.q_nope, c.q_rope, c.ckv, c.k, c.table, c.query_start, c.key_length)]
    for given in (True, False):
        out = torch.zeros_like(args[0])
        call = kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale)
        at, size = call.workspace.data_ptr(), call.workspace.numel()
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            torch.cuda._sleep(100_000_000)   # tens of milliseconds
            if not given:
                call()
        if given:
            call(st)
        del call
        others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert not st.query(), "the stream was done too early for this test"
        assert all(o.data_ptr() != at for o in others)
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), ref[0])
        del others


def test_bound_calls_follow_their_buffers():
    g = torch.Generator().manual_seed(5)
    q = torch.randn(4, 8, 64, generator=g).bfloat16().cuda()
    pos = torch.arange(4, device="cuda")
    out = torch.zeros_like(q)
    call = kvr.prepare_query_rope(q, pos, out)
    for seed in (1, 2):
        q.copy_(torch.randn(4, 8, 64, generator=torch.Generator().manual_seed(seed)))
        call()
        want = torch.zeros_like(q)
        kvr.query_rope(q, pos, want)
        assert torch.equal(out, want)
    with pytest.raises(TypeError):
        call.staged(0, 0, 0)


def test_workspace_given():
    c = mla_case([2, 1], [300, 90], 8, seed=23)
    ref = run_mla(c)
    d = lambda t: t.cuda()  # noqa: E731
    args = [d(t).contiguous() for t in (c.q_nope, c.q_rope, c.ckv, c.k, c.table, c.query_start, c.key_length)]
    out = torch.zeros_like(args[0])
    need = kvr.prepare_mla_attention(*args, out, softmax_scale=c.scale).workspace.numel()
    ws = torch.full((need,), 0xFF, device="cuda", dtype=torch.uint8)   # its contents do not matter
    kvr.mla_attention(*args, out, softmax_scale=c.scale, workspace=ws)
    assert np.array_equal(out.double().cpu().numpy(), ref[0])
    for bad in (ws[:need - 1], ws[8:]):
        with pytest.raises(kvr.KvrError) as e:
            kvr.mla_attention(*args, out, softmax_scale=c.scale, workspace=bad)
        assert e.value.code == N.KVR_ERR_SHAPE
    with pytest.raises(kvr.KvrError) as e:
        kvr.mla_attention(*args, out, softmax_scale=c.scale, workspace=args[2].view(-1).view(torch.uint8))
    assert e.value.code in (N.KVR_ERR_ALIAS, N.KVR_ERR_SHAPE)


@pytest.mark.parametrize("pad,dtype", [(8, "bf16"), (16, "f16"), (64, "bf16")])
def test_strided_output(pad, dtype):
    """Rows of out in a wider tensor, heads and tokens in either order; the rest stays."""
    c = mla_case([2, 3], [150, 99], 5, dtype=dtype, seed=24)
    ref = run_mla(c)
    d = lambda t: t.cuda()  # noqa: E731
    args = [d(t) for t in (c.q_nope.contiguous(), c.q_rope.contiguous(), c.ckv, c.k, c.table, c.query_start, c.key_length)]
    for swap in (False, True):
        wide = torch.full((5, 5, DV + pad), SENTINEL, device="cuda", dtype=args[0].dtype)
        out = (wide.transpose(0, 1) if swap else wide)[..., :DV]
        kvr.mla_attention(*args, out, softmax_scale=c.scale)
        assert np.array_equal(out.double().cpu().numpy(), ref[0])
        assert (wide[..., DV:] == SENTINEL).all()


def test_nothing_is_read_of_holes_and_behind_the_last_key():
    """NaN in the blocks that the table leaves out, in those that no entry names and in a block's rows behind the last key."""
    c = mla_case([1, 4], [200, 90], 16, block_size=32, seed=25)
    held = c.table[0, 3].clone(), c.table[1, 1].clone()
    c.table[0, 3] = c.table[1, 1] = -1
    for h in held:
        c.ckv[h] = float("nan")
        c.k[h] = float("nan")
    check_mla(c, run_mla(c), oracle_mla(c))


def test_a_shared_prefix_and_the_same_sequence_twice():
    """Blocks that several sequences name (and one names twice)."""
    c = mla_case([1, 1, 2], [100, 100, 100], 8, block_size=32, seed=26)
    c.table[1] = c.table[0]
    c.table[2, 0] = c.table[2, 1] = c.table[0, 0]
    check_mla(c, run_mla(c), oracle_mla(c))


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_odd_softmax_scales(scale):
    check_mla(mla_case([2], [130], 8, scale=scale, seed=27), run_mla(mla_case([2], [130], 8, scale=scale, seed=27)),
              oracle_mla(mla_case([2], [130], 8, scale=scale, seed=27)))


def test_extreme_scales_of_codes():
    """1 / scale over 40 octaves and queries far from 1: halves neither overflow nor lose the score."""
    c = mla_case([2, 1], [90, 40], 6, cache="int8", scale_len=0, seed=28)
    c.ckv_scale = c.ckv_scale * 2.0 ** 20
    c.q_nope = (c.q_nope.float() * 2.0 ** 18).to(c.q_nope.dtype)
    got, want = run_mla(c), oracle_mla(c)
    assert np.isfinite(got[0]).all()
    assert np.linalg.norm(got[0] - want[0]) <= 2.0 ** -6 * np.linalg.norm(want[0])
    c.ckv_scale = c.ckv_scale * 2.0 ** -44
    c.q_nope = (c.q_nope.float() * 2.0 ** -44).to(c.q_nope.dtype)
    got, want = run_mla(c), oracle_mla(c)
    assert np.linalg.norm(got[0] - want[0]) <= 2.0 ** -6 * np.linalg.norm(want[0])


def test_mla_refusals():
    c = mla_case([2, 1], [60, 40], 4, seed=29)
    d = lambda t: t.cuda()  # noqa: E731
    base = dict(q_nope=d(c.q_nope).contiguous(), q_rope=d(c.q_rope).contiguous(), ckv_cache=d(c.ckv), k_cache=d(c.k), block_table=d(c.table),
                query_start=d(c.query_start), key_length=d(c.key_length), out=torch.zeros(c.q_nope.shape, device="cuda", dtype=torch.bfloat16),
                softmax_scale=0.1)
    bad = [dict(q_nope=base["q_nope"].float()), dict(q_rope=base["q_rope"][:2]), dict(q_rope=base["q_rope"].half()),
           dict(out=base["out"].half()), dict(out=base["out"][:, :3]), dict(block_table=None), dict(block_table=base["block_table"].int()),
           dict(block_table=base["block_table"][:1]), dict(block_table=base["block_table"].t()), dict(query_start=base["query_start"][:2]),
           dict(key_length=base["key_length"].int()), dict(k_cache=base["k_cache"][:1]), dict(cache_mode="Norm"), dict(cache_mode="x"),
           dict(ckv_cache=base["ckv_cache"].half()), dict(q_nope=base["q_nope"][..., :256]), dict(lse=torch.zeros(3, 4, device="cuda").double()),
           dict(lse=torch.zeros(3, 5, device="cuda")), dict(dev_status=torch.zeros(1, device="cuda")), dict(q_nope=base["q_nope"].cpu()),
           dict(key_length=base["key_length"].cpu()), dict(ckv_scale=torch.ones(3, device="cuda"))]
    for kw in bad:
        a = dict(base)
        a.update(kw)
        args = [a.pop(k) for k in ("q_nope", "q_rope", "ckv_cache", "k_cache", "block_table", "query_start", "key_length", "out")]
        with pytest.raises(ValueError):
            kvr.mla_attention(*args, **a)
    for kw in (dict(ckv_scale=torch.ones(1, device="cuda")), dict(ckv_cache=base["ckv_cache"].to(torch.int8)), dict(softmax_scale=float("nan")),
               dict(out=base["q_nope"])):
        a = dict(base)
        a.update(kw)
        args = [a.pop(k) for k in ("q_nope", "q_rope", "ckv_cache", "k_cache", "block_table", "query_start", "key_length", "out")]
        with pytest.raises(kvr.KvrError):
            kvr.mla_attention(*args, **a)
    assert (base["out"] == 0).all()
