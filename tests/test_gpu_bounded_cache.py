"""The operators as a serving loop uses them: a drafted tree verified, its accepted branch moved behind the context, the keys'
weights added up, the cache cut by them, and attention over what stays, against the float64 oracle step by step."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
import oracle
from cache_helpers import parents
from helpers import f64

pytestmark = pytest.mark.gpu

H, DV, DK, BS, BLOCKS, SCALE = 8, 512, 64, 16, 40, 0.0722


class Loop:
    """Three conversations of other lengths over one paged cache."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
        i = lambda x: torch.tensor(x, dtype=torch.int64).cuda()  # noqa: E731
        self.new, keys = [9, 5, 12], [120, 40, 75]
        T = sum(self.new)
        self.ckv, self.k = r(BLOCKS, BS, 1, DV).cuda(), r(BLOCKS, BS, 1, DK).cuda()
        self.table = torch.randperm(BLOCKS, generator=g)[:30].view(3, 10).cuda()
        self.q, self.pe = r(T, H, DV).cuda(), r(T, H, DK).cuda()
        self.start, self.length = i([0, 9, 14, 26]), i(keys)
        self.parent = parents(self.new, 4).cuda()
        self.mask, self.positions = torch.zeros(T, 1, dtype=torch.int64, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
        self.turned, self.out, self.lse = torch.zeros_like(self.pe), torch.zeros_like(self.q), torch.zeros(T, H, device="cuda")
        # the branch that the sampler accepted, and its queries beside one another
        self.before = i([k - n for k, n in zip(keys, self.new)])
        branch, rows = [], []
        for n, words in enumerate([oracle.cache_ops.ancestors(self.parent.tolist()[a:b]) for a, b in ((0, 9), (9, 14), (14, 26))]):
            path = sorted(words[-1])
            branch.append(path)
            rows += [sum(self.new[:n]) + x for x in path]
        most = max(map(len, branch))
        self.accepted = i([[keys[n] - self.new[n] + x for x in path] + [-1] * (most - len(path)) for n, path in enumerate(branch)])
        self.count, self.rows = i([len(path) for path in branch]), i(rows)
        self.start2 = i([0] + list(np.cumsum([len(path) for path in branch])))
        self.length2 = self.before + self.count
        self.weight = torch.zeros(3, 160, device="cuda")
        self.q2, self.pe2, self.lse2 = (torch.zeros_like(x[: len(rows)]) for x in (self.q, self.pe, self.lse))
        self.kept, self.kept_length = torch.zeros(3, 64, dtype=torch.int64, device="cuda"), i([0, 0, 0])
        self.next = torch.zeros(3, 160, device="cuda")
        self.last = i([0, 1, 2, 3])
        self.q3, self.pe3, self.out3 = r(3, H, DV).cuda(), r(3, H, DK).cuda(), torch.zeros(3, H, DV, dtype=torch.bfloat16, device="cuda")

    def step(self):
        kvr.draft_tree(self.parent, self.start, self.mask, position_start=self.before, positions=self.positions)
        kvr.query_rope(self.pe, self.positions, self.turned)
        kvr.mla_attention(self.q, self.turned, self.ckv, self.k, self.table, self.start, self.length, self.out, softmax_scale=SCALE,
                          lse=self.lse, tree_mask=self.mask)
        kvr.kv_cache_compact(self.ckv, self.k, self.table, self.accepted, self.count, start=self.before)
        torch.index_select(self.q, 0, self.rows, out=self.q2)
        torch.index_select(self.turned, 0, self.rows, out=self.pe2)
        torch.index_select(self.lse, 0, self.rows, out=self.lse2)
        kvr.mla_key_weight(self.q2, self.pe2, self.ckv, self.k, self.table, self.start2, self.length2, self.lse2, self.weight,
                           softmax_scale=SCALE, past=self.weight)
        kvr.kv_cache_select(self.weight, self.length2, self.kept, self.kept_length, sink=2, recent=8, kept_weight=self.next)
        kvr.kv_cache_compact(self.ckv, self.k, self.table, self.kept, self.kept_length)
        kvr.mla_attention(self.q3, self.pe3, self.ckv, self.k, self.table, self.last, self.kept_length, self.out3, softmax_scale=SCALE)

    def results(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.mask, self.positions, self.out, self.lse, self.weight, self.kept, self.kept_length, self.next,
                                    self.ckv, self.k, self.out3)]


def test_a_loop_against_the_oracle():
    s = Loop()
    n = lambda t: t.cpu().numpy()  # noqa: E731
    ckv, k = f64(s.ckv)[:, :, 0].copy(), f64(s.k)[:, :, 0].copy()
    s.step()
    mask, pos, out, lse, weight, kept, count, carried, gv, gk, out3 = s.results()
    rm, rp = np.zeros(mask.shape, dtype=np.int64), np.zeros(pos.shape, dtype=np.int64)
    assert oracle.ref_draft_tree(n(s.parent), n(s.start), rm, n(s.before), rp) == 0
    assert np.array_equal(n(mask), rm) and np.array_equal(n(pos), rp)
    ro, rl = np.zeros(out.shape), np.zeros(lse.shape)
    scale = float(np.float32(SCALE))
    oracle.ref_mla_tree_attention(f64(s.q), f64(s.turned), ckv, k, n(s.table), n(s.start), n(s.length), rm, ro, rl, scale=scale)
    # a weight and the output are rounded to bf16, 2^-8 each; scores are off by 2^-17 of terms of about 30 in all
    assert np.abs(f64(out) - ro).max() <= (2.0 ** -7 + 2.0 ** -11) * np.abs(ro).max() + 2.0 ** -7 * np.abs(ckv).max() * 0.25
    assert np.abs(f64(lse) - rl).max() <= 2.0 ** -11
    # the branch that was accepted is a causal chain: each token's weights add up to one a head
    assert oracle.ref_kv_cache_compact(ckv, k, n(s.table), n(s.accepted), n(s.count), n(s.before)) == 0
    rw = np.zeros(weight.shape)
    oracle.ref_mla_key_weight(f64(s.q2), f64(s.pe2), ckv, k, n(s.table), n(s.start2), n(s.length2), f64(s.lse2), rw, scale=scale)
    assert np.allclose(f64(weight), rw, rtol=2.0 ** -10, atol=1e-30)
    assert np.allclose(f64(weight).sum(1), H * n(s.count), rtol=2.0 ** -9)
    st, rk, rc, rn = oracle.ref_kv_cache_select(n(weight), n(s.length2), 64, 2, 8)
    assert st == 0 and np.array_equal(n(kept), rk) and np.array_equal(n(count), rc) and np.array_equal(n(carried)[:, :64], rn)
    assert oracle.ref_kv_cache_compact(ckv, k, n(s.table), rk, rc) == 0
    assert np.array_equal(f64(gv)[:, :, 0], ckv) and np.array_equal(f64(gk)[:, :, 0], k)
    ro = np.zeros(out3.shape)
    oracle.ref_mla_attention(f64(s.q3), f64(s.pe3), ckv, k, n(s.table), n(s.last), rc, ro, np.zeros((3, H)), scale=scale)
    assert np.abs(f64(out3) - ro).max() <= (2.0 ** -7 + 2.0 ** -11) * np.abs(ro).max() + 2.0 ** -7 * np.abs(ckv).max() * 0.25


def test_the_loop_in_a_graph_and_on_a_side_stream():
    want = Loop(1)
    want.step()
    want = want.results()
    s = Loop(1)
    keep = [x.clone() for x in (s.ckv, s.k)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    assert all(torch.equal(a, b) for a, b in zip(want, s.results()))
    s = Loop(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for _ in range(2):
        s.ckv.copy_(keep[0])
        s.k.copy_(keep[1])
        s.weight.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, s.results()))
