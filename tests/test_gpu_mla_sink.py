"""mla_attention where one key has nearly all the weight and many keys far below it carry the output (an attention sink,
whose value is small): weights that are rounded to halves keep them.

All rows have the same query, so that one row in float64 is the oracle of all; with as many row tiles as CTA pairs, or
more, each pair goes over all keys of its rows."""
import math

import pytest
import torch

import attention_prologue_kv_gb300 as kvr
from attention_helpers import DTYPES, half_step

pytestmark = pytest.mark.gpu

N, T, H, BS = 1 << 17, 80, 128, 128


def sink_case(dtype, cache, octaves, at):
    """N keys `octaves` below the one at place `at`; the rotary part alone makes the scores. A value's mean is 1/2."""
    g = torch.Generator("cuda").manual_seed(3)
    dt = DTYPES[dtype]
    c = (0.5 + 0.25 * torch.randn(N, 512, generator=g, device="cuda")).clamp(-1, 2)
    c[at] = 0
    scale = None
    if cache == "int8":
        scale = torch.full((1,), 60.0, device="cuda")
        c = (c * 60).round()
    ckv = c.to(DTYPES[cache or dtype]).view(-1, BS, 1, 512)
    k = torch.zeros(N, 64, device="cuda", dtype=dt)
    k[:, 0] = -octaves
    k[at, 0] = 0
    q_rope = torch.zeros(1, 1, 64, device="cuda", dtype=dt)
    q_rope[..., 0] = 1
    table = torch.arange(N // BS, device="cuda").view(1, -1)
    return dict(q_nope=torch.zeros(1, 1, 512, device="cuda", dtype=dt).expand(T, H, 512), q_rope=q_rope.expand(T, H, 64), ckv=ckv,
                k=k.view(-1, BS, 1, 64), table=table, scale=scale)


def run(c):
    out = torch.full((T, H, 512), -77.0, device="cuda", dtype=c["q_nope"].dtype)
    lse = torch.full((T, H), -77.0, device="cuda")
    kvr.mla_attention(c["q_nope"], c["q_rope"], c["ckv"], c["k"], c["table"], torch.tensor([0, T], device="cuda"),
                      torch.tensor([N], device="cuda"), out, softmax_scale=math.log(2.0), causal=False, ckv_scale=c["scale"], lse=lse)
    return out.double(), lse.double()


def oracle(c):
    """(out [512], sum of |weight * value| [512], lse) of the row."""
    s = float(torch.tensor(math.log(2.0), dtype=torch.float32)) * c["k"].view(N, 64)[:, 0].double()
    v = c["ckv"].view(N, 512).double()
    v = v if c["scale"] is None else v / c["scale"].double()
    p = torch.softmax(s, 0)
    return p @ v, p @ v.abs(), torch.logsumexp(s, 0)


@pytest.mark.parametrize("at", [0, 70000, N - 1])
@pytest.mark.parametrize("octaves", [18.0, 23.375, 25.25])   # below 2^-14, near the last bit, below the last half
@pytest.mark.parametrize("dtype,cache", [("f16", None), ("f16", "int8"), ("bf16", "int8"), ("bf16", None)])
def test_the_keys_below_a_sink(dtype, cache, octaves, at):
    """To first order, with u = half a step of the weights' type: each weight is off by u of itself and, as a half, by 2^-32
    of the largest weight (2^-25, half of a half's last step, 7 octaves up), which is at most 1 of the sum; the score of
    exact products by 2^-21; float32 sums of the output take 16 keys an addition and of the weights 2 keys an addition in
    four threads, each addition off by at most 2^-23: N (2^-27 + 2^-26); the output is rounded once."""
    c = sink_case(dtype, cache, octaves, at)
    out, lse = run(c)
    want, size, want_lse = oracle(c)
    halves = dtype == "f16" or cache is not None
    u_weight = 2.0 ** -11 if halves else 2.0 ** -8
    u_out = half_step(DTYPES[dtype])
    mean = c["ckv"].view(N, 512).double().abs().mean(0) / (60.0 if cache else 1.0)
    tol = u_out * want.abs() + (u_weight + 2.0 ** -20 + N * (2.0 ** -27 + 2.0 ** -26)) * size + (N * 2.0 ** -32 * mean if halves else 0)
    if dtype == "f16":
        tol = tol + 2.0 ** -25
    off = (out - want).abs()
    assert (off <= tol * (1 + 2.0 ** -6)).all(), "off by up to %.3g of the output" % float((off / want.abs()).max())
    assert float((lse - want_lse).abs().max()) <= 2.0 ** -20 + N * 2.0 ** -26 + 2.0 ** -24 * abs(float(want_lse))


@pytest.mark.parametrize("octaves", [22.5, 23.375, 24.25])   # about 3, 1.5 and 1 of a float32's last place, two at a time
@pytest.mark.parametrize("dtype,cache", [("f16", None), ("bf16", "int8"), ("bf16", None)])
def test_the_sum_beside_a_sink(dtype, cache, octaves):
    """Equal small weights round to the same side each time they are added to the sink's: a thread adds its part of a step
    of 64 keys at once, N / 64 additions of 2^-24 of the sum each."""
    c = sink_case(dtype, cache, octaves, 5)
    _, lse = run(c)
    want = float(oracle(c)[2])
    assert float((lse - want).abs().max()) <= 2.0 ** -20 + N * 2.0 ** -30 + 2.0 ** -24 * abs(want)


@pytest.mark.parametrize("octaves", [22.5, 23.375, 24.25])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_the_plain_kernel_beside_a_sink(dtype, octaves):
    """Rows of 10 + 6 channels, a few of them: 64 keys are summed before they join the long sums, N / 64 additions of 2^-24
    each in the sum of the weights and in the output's, 64 within a block; the sink has a value here too. A weight is
    2^-20 off (two roundings of its score, expf)."""
    dt = DTYPES[dtype]
    c = sink_case(dtype, None, octaves, 5)
    c["ckv"] = c["ckv"][..., :10].contiguous()
    c["ckv"].view(N, 10)[5] = 1
    c["k"] = c["k"][..., :6].contiguous()
    c["q_nope"], c["q_rope"] = c["q_nope"][:2, :3, :10], c["q_rope"][:2, :3, :6]
    out, lse = torch.zeros(2, 3, 10, device="cuda", dtype=dt), torch.zeros(2, 3, device="cuda")
    call = kvr.prepare_mla_attention(c["q_nope"], c["q_rope"], c["ckv"], c["k"], c["table"], torch.tensor([0, 2], device="cuda"),
                                     torch.tensor([N], device="cuda"), out, softmax_scale=math.log(2.0), causal=False, lse=lse)
    assert call.workspace is None
    call()
    s = float(torch.tensor(math.log(2.0), dtype=torch.float32)) * c["k"].view(N, 6)[:, 0].double()
    p, v = torch.softmax(s, 0), c["ckv"].view(N, 10).double()
    want, size, want_lse = p @ v, p @ v.abs(), float(torch.logsumexp(s, 0))
    rel = 2.0 ** -19 + N * 2.0 ** -30 + 64 * 2.0 ** -24
    assert ((out.double() - want).abs() <= half_step(dt) * want.abs() * (1 + 2.0 ** -6) + 2 * rel * size).all()
    assert float((lse.double() - want_lse).abs().max()) <= rel + 2.0 ** -23 * abs(want_lse)


def unit_scale():
    """The softmax scale whose float32 product with log2(e) is 1: scores in octaves are the products themselves."""
    log2e = torch.tensor(1.4426950408889634, dtype=torch.float32)
    x = torch.tensor(math.log(2.0), dtype=torch.float32)
    near = [torch.nextafter(x, x - 1), x, torch.nextafter(x, x + 1)]
    return next(float(v) for v in near if float(v * log2e) == 1.0)


@pytest.mark.parametrize("base", [10, 23, 24, 25, 26, 28])
@pytest.mark.parametrize("dtype,cache", [("f16", None), ("f16", "int8"), ("bf16", "int8"), ("bf16", None)])
def test_scores_that_a_float_holds_coarsely(dtype, cache, base):
    """Scores of 2^base octaves and 0 to 12 above, in multiples of what a float32 of that size can tell apart: the first step's
    keys set the reference, later ones are up to 8 octaves above it and then more."""
    unit, n = 2.0 ** max(base - 23, 0), 512
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(base)
    above = torch.zeros(n)
    above[64:128] = (torch.randint(0, 9, (64,), generator=g) / unit).floor() * unit
    above[128:] = (torch.randint(0, 13, (n - 128,), generator=g) / unit).floor() * unit
    k = torch.zeros(n, 64)
    k[:, 0], k[:, 1] = 2.0 ** (base // 2), above
    q_rope = torch.zeros(64)
    q_rope[0], q_rope[1] = 2.0 ** (base - base // 2), 1
    v = torch.randn(n, 512, generator=g)
    scale = None
    if cache:
        v, scale = (v * 20).round().clamp(-128, 127), torch.full((1,), 20.0, device="cuda")
    c = dict(ckv=v.to(DTYPES[cache or dtype]).cuda().view(4, 128, 1, 512), k=k.to(dt).cuda().view(4, 128, 1, 64))
    assert torch.equal(c["k"].float().cpu().view(n, 64), k)
    rows = 70   # both CTAs of a pair
    out, lse = torch.zeros(1, rows, 512, device="cuda", dtype=dt), torch.zeros(1, rows, device="cuda")
    kvr.mla_attention(torch.zeros(1, rows, 512, device="cuda", dtype=dt), q_rope.to(dt).cuda().expand(1, rows, 64).contiguous(), c["ckv"],
                      c["k"], torch.arange(4, device="cuda").view(1, 4), torch.tensor([0, 1], device="cuda"), torch.tensor([n], device="cuda"),
                      out, softmax_scale=unit_scale(), ckv_scale=scale, lse=lse)
    p = torch.softmax(above.double().cuda() * math.log(2.0), 0)
    value = c["ckv"].view(n, 512).double() / (20.0 if cache else 1.0)
    want, size = p @ value, p @ value.abs()
    # Differences of scores are exact and whole, so weights are powers of two and round nowhere; 512 keys in float32.
    assert ((out.double() - want).abs() <= half_step(dt) * want.abs() * (1 + 2.0 ** -6) + 2.0 ** -14 * size).all()
    want_lse = (2.0 ** base + torch.logsumexp(above.double() * math.log(2.0), 0) / math.log(2.0)) * math.log(2.0)
    assert float((lse.double() - float(want_lse)).abs().max()) <= 2.0 ** -22 * float(want_lse)
