"""GPU parity of kv_cache_read against the float64 oracle: 16-bit rows bit for
bit; an 8-bit code's value is the code times 1/scale, each rounded to float32
(2 x 2^-24), then to the type (u)."""
import numpy as np
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
import oracle
from attention_helpers import DTYPES, cache_values, half_step
from helpers import f64, guarded

pytestmark = pytest.mark.gpu


def check(B, S, mode, Dv=512, Dk=64, block=16, dtype="bf16", cache=None, k_cache=None, per_channel=True, pad=0, seed=0, bad=False):
    g = torch.Generator().manual_seed(seed)
    cache, k_cache, dt = cache or dtype, k_cache or dtype, DTYPES[dtype]
    if mode == "Norm":
        d0, d1 = B + 1, block
        index = torch.randint(0, d1, (B, S), generator=g)
    elif mode == "PA_BSND":
        d0, d1 = 7, block
        index = torch.randint(0, d0 * d1, (B * S,), generator=g)
    else:
        d0, d1 = 9, block
        nblk = -(-S // d1)
        last = S - (nblk - 1) * d1
        index = torch.randint(0, d0, (B, nblk), generator=g) * d1
        if last < d1:   # an entry inside its block
            index[:, -1] += torch.randint(0, d1 - last + 1, (B,), generator=g)
        index = index.reshape(-1)
    flat = index.view(-1)
    flat[torch.rand(flat.shape, generator=g) < 0.1] = -1
    if bad:
        flat[0] = d0 * d1 if mode != "Norm" else d1
        flat[-1] = -2
    ckv, cs = cache_values(g, (d0, d1, 1, Dv), cache, Dv if per_channel else 1)
    k, ks = cache_values(g, (d0, d1, 1, Dk), k_cache, Dk if per_channel else 1)
    out, c1 = guarded((B, 1, S, Dv + Dk + pad), dt, -9.0)
    view = out[..., :Dv + Dk]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.kv_cache_read(ckv.cuda(), k.cuda(), index.cuda(), view, cache_mode=mode, ckv_scale=None if cs is None else cs.cuda(),
                      k_scale=None if ks is None else ks.cuda(), dev_status=st)
    torch.cuda.synchronize()
    c1()
    want = np.full((B, S, Dv + Dk), -9.0)
    rst = oracle.ref_kv_cache_read(want, f64(ckv)[:, :, 0], f64(k)[:, :, 0], index.numpy(), mode,
                                   None if cs is None else f64(cs), None if ks is None else f64(ks))
    got = f64(out)[:, 0]
    assert (got[..., Dv + Dk:] == -9).all()
    got = got[..., :Dv + Dk]
    assert int(st.item()) == rst == (1 if bad else 0)
    u = half_step(dt)
    for part, scale in ((slice(0, Dv), cs), (slice(Dv, Dv + Dk), ks)):
        w, x = want[..., part], got[..., part]
        if scale is None:
            assert np.array_equal(w, x)
        else:
            assert (np.abs(x - w) <= (u * (1 + 2.0 ** -20) + 2.0 ** -22) * np.abs(w) + float(torch.finfo(dt).tiny) * 2.0 ** -9).all()


@pytest.mark.parametrize("mode", ["Norm", "PA_BSND", "PA_BLK_BSND"])
@pytest.mark.parametrize("B,S,block", [(1, 1, 1), (3, 37, 64), (2, 130, 48), (5, 7, 33), (300, 1, 16)])
def test_modes(mode, B, S, block):
    check(B, S, mode, block=block, seed=S)


@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cache", ["int8", "fp8_e4m3fn", "fp8_e5m2"])
@pytest.mark.parametrize("k8", [True, False])
def test_codes(cache, dtype, per_channel, k8):
    check(2, 33, "PA_BSND", dtype=dtype, cache=cache, k_cache=cache if k8 else None, per_channel=per_channel, seed=5)


@pytest.mark.parametrize("Dv,Dk,pad", [(1, 1, 0), (10, 6, 0), (256, 32, 8), (520, 72, 3), (1032, 8, 0), (512, 64, 64), (24, 8, 1)])
@pytest.mark.parametrize("cache", [None, "int8"])
def test_widths(Dv, Dk, pad, cache):
    check(2, 9, "PA_BSND", Dv, Dk, cache=cache, pad=pad, seed=Dv)


@pytest.mark.parametrize("mode", ["Norm", "PA_BSND", "PA_BLK_BSND"])
def test_bad_entries_leave_their_rows(mode):
    check(2, 33, mode, block=40 if mode == "Norm" else 16, bad=True)


def test_every_code_decodes_exactly():
    """All 256 codes of each type at scale 1 (NaN codes to NaN)."""
    for name in ("int8", "fp8_e4m3fn", "fp8_e5m2"):
        codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(DTYPES[name]).view(1, 1, 1, 256).cuda()
        k = torch.zeros(1, 1, 1, 8, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros(1, 264, dtype=torch.bfloat16, device="cuda")
        kvr.kv_cache_read(codes, k, torch.zeros(1, dtype=torch.int64, device="cuda"), out, ckv_scale=torch.ones(1, device="cuda"))
        want = codes.view(-1).cpu().to(torch.float32)
        got = out[0, :256].cpu().to(torch.float32)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~want.isnan()], want[~want.isnan()])


def test_refusals():
    ckv = torch.zeros(2, 4, 1, 16, device="cuda", dtype=torch.bfloat16)
    k, out = torch.zeros(2, 4, 1, 8, device="cuda", dtype=torch.bfloat16), torch.zeros(3, 24, device="cuda", dtype=torch.bfloat16)
    index = torch.zeros(3, device="cuda", dtype=torch.int64)
    s = torch.ones(16, device="cuda")
    bad = [dict(index=index[:2]), dict(index=index.int()), dict(out=out[:, :20]), dict(out=out.half()), dict(out=out.cpu()),
           dict(cache_mode="PA"), dict(k_cache=k[:1]), dict(ckv_scale=s[:3]), dict(ckv_scale=s.double()), dict(index=index.cpu()),
           dict(dev_status=torch.zeros(1, device="cuda"))]
    for kw in bad:
        a = dict(ckv_cache=ckv, k_cache=k, index=index, out=out)
        a.update(kw)
        with pytest.raises(ValueError):
            kvr.kv_cache_read(a.pop("ckv_cache"), a.pop("k_cache"), a.pop("index"), a.pop("out"), **a)
    for kw in (dict(ckv_scale=s), dict(ckv_cache=ckv.to(torch.int8)), dict(out=ckv.view(8, 16)[:3].as_strided((3, 24), (24, 1)))):
        a = dict(ckv_cache=ckv, k_cache=k, index=index, out=out)
        a.update(kw)
        with pytest.raises(kvr.KvrError):
            kvr.kv_cache_read(a.pop("ckv_cache"), a.pop("k_cache"), a.pop("index"), a.pop("out"), **a)
