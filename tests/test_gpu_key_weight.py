"""mla_key_weight against the float64 oracle."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
from attention_helpers import SENTINEL, mla_case
from cache_helpers import check_weight, cuda, oracle_weight, queries, row_lse, run_weight
from helpers import f64

pytestmark = pytest.mark.gpu


def width_of(c, more=3):
    return int(c.key_length.max()) + more


def check(c, lse=None, **kw):
    lse = row_lse(c) if lse is None else lse
    width = width_of(c)
    gpu = run_weight(c, lse, width, **kw)
    kw.pop("pad", None)
    kw.pop("stream", None)
    ref = oracle_weight(c, lse, width, **kw)
    check_weight(c, gpu, ref, kw.get("past"), kw.get("decay", 1.0))
    return gpu


@pytest.mark.parametrize("kw", [
    dict(new=[1], keys=[1], H=1),
    dict(new=[1], keys=[1000], H=16, dtype="f16", block_size=128),
    dict(new=[1] * 9, keys=[1, 7, 128, 129, 255, 256, 257, 600, 31], H=128, block_size=128),
    dict(new=[1] * 40, keys=list(range(3, 43)), H=20, block_size=16),
    dict(new=[7, 1, 33, 0, 2], keys=[500, 1, 33, 8, 90], H=24, block_size=64),
    dict(new=[40, 3], keys=[300, 700], H=128, block_size=32),
    dict(new=[300], keys=[300], H=16, block_size=128),
    dict(new=[65, 130], keys=[700, 130], H=3, block_size=100),
    dict(new=[40], keys=[90], H=5, block_size=1),
    dict(new=[19, 2, 50], keys=[400, 33, 91], H=12, mode="Norm"),
    dict(new=[21], keys=[333], H=32, Dv=256, Dk=32, pad=8, block_size=64),
    dict(new=[5, 1], keys=[333, 64], H=32, Dv=448, Dk=64, block_size=64),
    dict(new=[9, 14], keys=[77, 130], H=3, Dv=70, Dk=6),
    dict(new=[2, 1], keys=[77, 30], H=3, Dv=600, Dk=64, dtype="f16"),
    dict(new=[2, 1], keys=[77, 30], H=2, Dv=1000, Dk=200)])
def test_sizes(kw):
    c = mla_case(seed=len(kw["new"]) + kw["H"], **kw)
    check(c)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,keys", [([30, 2], [30, 900]), ([50, 20], [30, 5]), ([128], [400])])
def test_causal_or_not(new, keys, causal):
    check(mla_case(new, keys, H=16, block_size=64, seed=3, causal=causal))


# Most tokens of a chunk see no key: the work that is cut is that of the others.
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,keys", [([1500, 700], [10, 300]), ([2100], [1]), ([3, 1300, 1], [40, 257, 5]), ([900, 4], [0, 9])])
def test_more_tokens_than_keys(new, keys, causal):
    check(mla_case(new, keys, H=16, block_size=64, seed=4, causal=causal))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache,k_cache,scale_len,k_scale_len", [
    ("int8", None, 1, 1), ("int8", None, 512, 1), ("fp8_e4m3fn", None, 512, 1), ("fp8_e5m2", None, 1, 1),
    ("fp8_e4m3fn", "fp8_e4m3fn", 1, 1), ("int8", "int8", 512, 64), ("fp8_e5m2", "int8", 1, 64), (None, "fp8_e4m3fn", 1, 64),
    (None, "int8", 1, 1)])
def test_codes(dtype, cache, k_cache, scale_len, k_scale_len):
    check(mla_case([1, 7, 40], [300, 90, 513], H=16, block_size=64, dtype=dtype, cache=cache, k_cache=k_cache, scale_len=scale_len,
                   k_scale_len=k_scale_len, seed=5))


@pytest.mark.parametrize("kw", [dict(block_size=16), dict(block_size=100), dict(block_size=1), dict(mode="Norm"),
                                dict(Dv=112, Dk=16), dict(Dv=512, Dk=48, block_size=64)])
def test_codes_in_other_blocks_and_widths(kw):
    scale_len = kw.get("Dv", 512)
    check(mla_case([1, 9], [300, 280], H=20, cache="fp8_e4m3fn", scale_len=scale_len, seed=6, **kw))


@pytest.mark.parametrize("kw", [dict(past=True), dict(past=True, decay=0.25), dict(past=True, decay=0.0), dict(past=True, in_place=True),
                                dict(past=True, in_place=True, decay=0.5, pad=5), dict(pad=3)])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 3]])
def test_past(new, kw):
    c = mla_case(new, [700, 129, 64], H=16, block_size=64, seed=7)
    kw = dict(kw)
    if kw.pop("past", False):
        kw["past"] = torch.rand(3, width_of(c), generator=torch.Generator().manual_seed(2)) * 20
    check(c, **kw)


def test_holes_get_nothing():
    c = mla_case([1, 20], [300, 200], H=16, block_size=16, seed=8, holes=[(0, 3), (0, 18), (1, 0)])
    past = torch.rand(2, width_of(c), generator=torch.Generator().manual_seed(3))
    gpu = check(c, past=past)
    assert np.array_equal(gpu[0][0, 48:64], f64(past)[0, 48:64])
    c.table[0, 5] = 10 ** 6      # out of range
    assert check(c)[1] == 1


def test_rows_of_infinite_lse():
    """-inf: a row that saw nothing adds nothing; +inf: its weights are zero; NaN reaches the keys that the row sees."""
    c = mla_case([30, 2], [200, 90], H=16, block_size=64, seed=9)
    lse = row_lse(c)
    lse[3, 2], lse[5], lse[31, 0] = -np.inf, -np.inf, np.inf
    check(c, lse)
    lse[0, 1] = np.nan
    w = run_weight(c, lse, width_of(c))[0]
    seen = 200 - 30 + 1
    assert np.isnan(w[0, :seen]).all() and not np.isnan(w[0, seen:200]).any() and not np.isnan(w[1]).any()


def test_a_key_that_is_not_finite_changes_its_own_weight_alone():
    for kw in (dict(H=16), dict(H=3, Dv=70, Dk=6)):
        c = mla_case([4, 1], [300, 100], block_size=64, seed=10, **kw)
        lse = row_lse(c)
        want = run_weight(c, lse, width_of(c))[0]
        e = int(c.table[0, 1])
        c.ckv[e, 5] = float("nan")
        c.ckv[e, 9, 0, 0] = float("inf")
        got = run_weight(c, lse, width_of(c))[0]
        others = np.ones(want.shape, dtype=bool)
        others[0, [69, 73]] = False
        assert np.isnan(got[0, 69]) and np.array_equal(got[others], want[others])


def test_lengths_that_are_left_out():
    c = mla_case([2, 3, 1, 4], [50, 60, 70, 80], H=8, block_size=16, seed=11, gap=3)
    lse, width = row_lse(c), width_of(c)
    for start, length, bits in (([0, 2, 5, 6, 10], [50, -1, 70, 80], 2), ([0, 2, 5, 6, 10], [50, 60, 10 ** 9, 80], 2),
                                ([0, 2, 1, 6, 10], [50, 60, 70, 80], 0x20), ([0, 2, 5, 6, 99], [50, 60, 70, 80], 0x20)):
        c.query_start, c.key_length = torch.tensor(start), torch.tensor(length)
        gpu, ref = run_weight(c, lse, width), oracle_weight(c, lse, width)
        check_weight(c, gpu, ref)
        assert gpu[1] & bits
    c.query_start, c.key_length = torch.tensor([0, 2, 5, 6, 10]), torch.tensor([50, 60, 70, 80])
    gpu, ref = run_weight(c, lse, 65), oracle_weight(c, lse, 65)   # no room for the last two sequences
    check_weight(c, gpu, ref)
    assert gpu[1] == 2 and (gpu[0][2:] == SENTINEL).all()


def test_far_positions_of_a_long_table():
    """Cache rows behind 2^31 elements, and few of many keys in a table with room for more."""
    d1, far = 128, 36000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 6 GB")
    c = mla_case([1, 5], [300, 513], H=16, block_size=d1, seed=12)
    big_v = torch.zeros(far + c.ckv.shape[0], d1, 1, 512, dtype=torch.bfloat16, device="cuda")
    big_k = torch.zeros(far + c.ckv.shape[0], d1, 1, 64, dtype=torch.bfloat16, device="cuda")
    big_v[far:], big_k[far:] = c.ckv.cuda(), c.k.cuda()
    table = torch.where(c.table < 0, -1, c.table + far)
    lse, w = row_lse(c), torch.zeros(2, 600, device="cuda")
    kvr.mla_key_weight(*queries(c), big_v, big_k, table.cuda(), cuda(c.query_start), cuda(c.key_length), lse.cuda(), w,
                       softmax_scale=c.scale)
    want = run_weight(c, lse, 600)[0]
    got = f64(w)
    for n, K in enumerate((300, 513)):
        assert np.array_equal(got[n, :K], want[n, :K])


def test_the_same_twice_captured_and_on_another_stream():
    for new, keys, H in (([1] * 5, [900, 31, 256, 700, 129], 16), ([200, 70], [900, 300], 32)):
        c = mla_case(new, keys, H=H, block_size=64, seed=13)
        lse, width = row_lse(c), width_of(c)
        want = run_weight(c, lse, width)[0]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        assert np.array_equal(run_weight(c, lse, width, stream=side)[0], want)
        w = torch.full((len(new), width), SENTINEL, device="cuda")
        call = kvr.prepare_mla_key_weight(*queries(c), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length),
                                          lse.cuda(), w, softmax_scale=c.scale)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(2):
            w.fill_(SENTINEL)
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(f64(w), want)


def test_refusals():
    c = mla_case([2], [20], H=4, seed=1)
    lse = row_lse(c)
    ok = dict(softmax_scale=c.scale)
    args = [*queries(c), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length)]
    w = torch.zeros(1, 24, device="cuda")
    for bad in ((None, w), (lse.cuda().double(), w), (lse.cuda()[:1], w), (lse.cuda(), w.double()), (lse.cuda(), w[0]),
                (lse.cuda(), torch.zeros(2, 24, device="cuda")), (lse.cuda(), torch.zeros(1, 48, device="cuda")[:, ::2]), (lse, w)):
        with pytest.raises(ValueError):
            kvr.mla_key_weight(*args, *bad, **ok)
    with pytest.raises(ValueError):
        kvr.mla_key_weight(*args, lse.cuda(), w, past=torch.zeros(1, 23, device="cuda"), **ok)
    two = torch.zeros(1, 40, device="cuda")
    with pytest.raises(kvr.KvrError):
        kvr.mla_key_weight(*args, lse.cuda(), two[:, :24], past=two[:, 8:32], **ok)


@pytest.mark.parametrize("kw", [dict(H=16), dict(H=40), dict(H=16, cache="int8"), dict(H=40, dtype="f16", cache="fp8_e4m3fn", scale_len=512),
                                dict(H=16, block_size=100), dict(H=3, Dv=70, Dk=6)])
def test_rows_of_others_do_not_matter(kw):
    """Queries of another sequence, and rows outside every sequence, share a group's products: NaN there stays there."""
    c = mla_case([3, 2, 7], [300, 500, 90], seed=14, gap=5, **dict(dict(block_size=64), **kw))
    lse, width = row_lse(c), width_of(c)
    want = run_weight(c, lse, width)[0]
    c.q_nope[12:] = float("nan")
    c.q_rope[12:] = float("inf")
    c.q_nope[3:5] = float("nan")
    got = run_weight(c, lse, width)[0]
    assert np.array_equal(got[[0, 2]], want[[0, 2]]) and np.isnan(got[1, :499]).all()


@pytest.mark.parametrize("new,keys,H", [([90], [100], 128), ([70, 3], [5000, 6000], 64), ([9] * 30, [700] * 30, 128),
                                        ([1] * 3, [9000, 20, 12000], 32), ([2] * 5, [3000] * 5, 128)])
def test_tiles_cut_over_many_ctas(new, keys, H):
    c = mla_case(new, keys, H=H, block_size=128, seed=15)
    check(c, past=torch.rand(len(new), width_of(c), generator=torch.Generator().manual_seed(5)))


def test_heads_that_share_a_query_and_strided_ones():
    """Expanded heads (stride 0), heads outside tokens, and rows with a gap between tokens."""
    c = mla_case([5, 30], [300, 200], H=8, block_size=64, seed=16)
    g = torch.Generator().manual_seed(1)
    for make in (lambda d: torch.randn(35, 1, d, generator=g).bfloat16().expand(35, 8, d),
                 lambda d: torch.randn(8, 35, d, generator=g).bfloat16().transpose(0, 1),
                 lambda d: torch.randn(35, 9, d, generator=g).bfloat16()[:, 1:]):
        qn, qr = make(512), make(64)
        c.q_nope, c.q_rope = qn.contiguous(), qr.contiguous()
        lse, w = row_lse(c), torch.full((2, 303), SENTINEL, device="cuda")
        on = lambda t: t._base.cuda().as_strided(t.shape, t.stride(), t.storage_offset())  # noqa: E731
        kvr.mla_key_weight(on(qn), on(qr), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length), lse.cuda(), w,
                           softmax_scale=c.scale)
        check_weight(c, (f64(w), 0), oracle_weight(c, lse, 303))


@pytest.mark.parametrize("kw", [dict(Dv=8, Dk=8), dict(Dv=8, Dk=8, block_size=4), dict(Dv=16, Dk=16, cache="int8", k_cache="int8"),
                                dict(Dv=16, Dk=8, cache="fp8_e5m2", block_size=16), dict(Dv=72, Dk=64, dtype="f16", mode="Norm"),
                                dict(Dv=136, Dk=24), dict(Dv=1, Dk=2), dict(Dv=336, Dk=64, cache="fp8_e4m3fn", scale_len=336)])
def test_narrow_rows(kw):
    check(mla_case([3, 20], [300, 77], H=11, scale=0.3, seed=17, **dict(dict(block_size=32), **kw)))


def test_more_heads_than_a_group():
    for H, new, keys in ((300, [1, 2], [513, 90]), (1000, [3], [700])):
        check(mla_case(new, keys, H=H, block_size=64, seed=18))


def test_two_calls_captured_on_branches_of_a_graph():
    both = [mla_case([3, 1], [900, 1500], H=24, block_size=64, seed=20), mla_case([40] * 3, [700] * 3, H=16, block_size=64, seed=21)]
    lses = [row_lse(c).cuda() for c in both]
    want = [run_weight(c, lse.cpu(), width_of(c))[0] for c, lse in zip(both, lses)]
    args = [[*queries(c), cuda(c.ckv), cuda(c.k), cuda(c.table), cuda(c.query_start), cuda(c.key_length)] for c in both]
    outs = [torch.full((len(c.key_length), width_of(c)), SENTINEL, device="cuda") for c in both]
    sides = [torch.cuda.Stream() for _ in both]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for side in sides:
            side.wait_stream(main)
        for a, lse, out, c, side in zip(args, lses, outs, both, sides):
            kvr.mla_key_weight(*a, lse, out, softmax_scale=c.scale, stream=side)
        for side in sides:
            main.wait_stream(side)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert np.array_equal(f64(out), w)
