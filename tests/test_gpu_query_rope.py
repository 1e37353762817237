"""GPU parity of query_rope against the float64 oracle.

Bound, u = half a step of the type: the rotation's two products and its sum
are float32 (3 roundings of 2^-24 of |a| + |b|), the angle's rest in half turns
is rounded once (2^-24 of at most 1, times pi) and sincospif is good to 2 units
in the last place: cos and sin are off by at most 2^-21, a value by at most
2^-20 (|a| + |b|), then rounded once (u |y|)."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
import oracle
from attention_helpers import DTYPES, half_step
from helpers import f64, guarded

pytestmark = pytest.mark.gpu


def check(T, H, D, sections, dtype="bf16", layout="interleave", base=10000.0, wide=0, tables=True, positions=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt, axes = DTYPES[dtype], len(sections)
    qw = torch.randn(T, H, wide + D, generator=g).to(dt)
    if positions is None:
        positions = torch.randint(-1000, 1 << 20, (axes, T), generator=g)
    q = qw.cuda()[..., wide:]
    out, c1 = guarded((T, H, D), dt, -3.0)
    cos, c2 = guarded((T, D), dt, -3.0)
    sin, c3 = guarded((T, D), dt, -3.0)
    kvr.query_rope(q, positions.cuda(), out, sections=sections, base=base, rope_layout=layout,
                   cos_out=cos if tables else None, sin_out=sin if tables else None)
    torch.cuda.synchronize()
    for c in (c1, c2, c3):
        c()
    q64 = f64(qw[..., wide:])
    want, wc, ws = oracle.ref_query_rope(q64, positions.numpy(), sections, base, layout == "half")
    u, tiny = half_step(dt), float(torch.finfo(dt).tiny) * 2.0 ** -3
    a, b = (q64[..., :D // 2], q64[..., D // 2:]) if layout == "half" else (q64[..., 0::2], q64[..., 1::2])
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    assert (np.abs(f64(out) - want) <= u * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -20 * size + tiny).all()
    if tables:
        for got, w in ((cos, wc), (sin, ws)):
            assert (np.abs(f64(got) - w) <= u * np.abs(w) * (1 + 2.0 ** -10) + 2.0 ** -20).all()
    else:
        assert (f64(cos) == -3).all()


@pytest.mark.parametrize("layout", ["interleave", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,D,sections,wide", [
    (1, 1, 64, [32], 0), (256, 128, 64, [32], 0), (37, 5, 64, [8, 12, 12], 128), (3, 9, 2, [1], 0),
    (7, 17, 48, [4, 0, 20], 8), (11, 2, 6, [1, 1, 1], 0), (5, 3, 20, [4, 3, 2, 1], 3), (2, 1, 256, [16] * 8, 0),
    (1031, 8, 128, [64], 0), (4, 130, 32, [16], 4)])
def test_shapes(T, H, D, sections, wide, dtype, layout):
    check(T, H, D, sections, dtype, layout, wide=wide, tables=(T + H) % 2 == 1, seed=T)


@pytest.mark.parametrize("base", [1.0, 10000.0, 1e6])
def test_far_positions(base):
    """The turns are dropped in fixed point. The oracle's own angle in float64 is
    good to |angle| 2^-52 (2^-21 at 2^31), so positions end there."""
    p = torch.tensor([[0, 1, -1, 2 ** 20, -2 ** 20 - 1, 2 ** 29 + 7, -2 ** 31]])
    check(7, 3, 64, [32], base=base, positions=p)
    check(7, 3, 64, [32], "f16", base=base, positions=p, layout="half")


def test_no_tokens_and_no_heads():
    kvr.query_rope(torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16), torch.empty(1, 0, device="cuda", dtype=torch.int64),
                   torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16))
    q = torch.empty(3, 0, 64, device="cuda", dtype=torch.bfloat16)
    cos, sin = torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16), torch.ones(3, 64, device="cuda", dtype=torch.bfloat16)
    kvr.query_rope(q, torch.zeros(3, device="cuda", dtype=torch.int64), torch.empty_like(q), cos_out=cos, sin_out=sin)
    assert (cos == 1).all() and (sin == 0).all()


def test_refusals():
    q = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    o, p = torch.zeros_like(q), torch.zeros(2, 4, device="cuda", dtype=torch.int64)
    bad = [dict(q=q.float()), dict(q=q[:, :, ::2]), dict(out=o[:3]), dict(out=o.half()), dict(positions=p.int()),
           dict(positions=p[:, :3]), dict(positions=p.t()), dict(sections=[32]), dict(sections=[31, 2]), dict(sections=None),
           dict(sections=[33, -1]), dict(rope_layout="last"), dict(cos_out=torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)),
           dict(positions=p.cpu()), dict(out=o.cpu())]
    for kw in bad:
        a = dict(q=q, positions=p, out=o, sections=[16, 16])
        a.update(kw)
        with pytest.raises(ValueError):
            kvr.query_rope(a.pop("q"), a.pop("positions"), a.pop("out"), **a)
    for kw in (dict(out=q), dict(base=0.5), dict(base=float("nan")), dict(out=o[:1].expand(4, 2, 64))):
        a = dict(q=q, positions=p, out=o, sections=[16, 16])
        a.update(kw)
        with pytest.raises(kvr.KvrError):
            kvr.query_rope(a.pop("q"), a.pop("positions"), a.pop("out"), **a)
    assert (o == 0).all()
