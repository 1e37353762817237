"""mla_attention where a part of a pair's work takes longer than the second after which a wait gives up."""
import pytest
import torch

import attention_prologue_kv_gb300 as kvr

pytestmark = pytest.mark.gpu


def test_a_part_of_more_than_a_second():
    """The most keys, in blocks of one, with codes in the rotary part: 5 us a step of 64 keys, 1.3 s a part, and the warps
    that bring a part's queries wait for all of the part before. (The table names 4096 rows over and over, so that the
    softmax is theirs; all rows (token, head) have the same query.)

    A part adds 16 keys at a time to an output's sum and a step to a thread's share of the weights' sum: 2^20 additions of
    2^-23 and 2^18 of 2^-24, of the weights' sum of magnitudes and of the sum."""
    keys, pool, T, H = 1 << 24, 1 << 12, 160, 128
    g = torch.Generator("cuda").manual_seed(60)
    ckv = torch.randn(pool, 1, 1, 512, generator=g, device="cuda").bfloat16()
    k = (torch.randn(pool, 1, 1, 64, generator=g, device="cuda") * 20).round().clamp(-128, 127).to(torch.int8)
    qn = torch.randn(1, 1, 512, generator=g, device="cuda").bfloat16().expand(T, H, 512)
    qr = torch.randn(1, 1, 64, generator=g, device="cuda").bfloat16().expand(T, H, 64)
    table = torch.arange(pool, device="cuda").repeat(keys // pool).view(1, -1)
    out, lse = torch.zeros(T, H, 512, device="cuda", dtype=torch.bfloat16), torch.zeros(T, H, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.mla_attention(qn, qr, ckv, k, table, torch.tensor([0, T], device="cuda"), torch.tensor([keys], device="cuda"), out,
                      softmax_scale=0.0722, causal=False, k_scale=torch.full((1,), 20.0, device="cuda"), lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    c, r = ckv.view(pool, 512).double(), k.view(pool, 64).double() / 20
    s = float(torch.tensor(0.0722, dtype=torch.float32)) * (c @ qn[0, 0].double() + r @ qr[0, 0].double())
    p = torch.softmax(s, 0)
    want, size, want_lse = p @ c, p @ c.abs(), float(torch.logsumexp(s, 0)) + 12 * 0.6931471805599453
    assert ((out.double() - want).abs() <= (2.0 ** -3 + 2.0 ** -7) * size).all()
    assert float((lse.double() - want_lse).abs().max()) <= 2.0 ** -6 + 2.0 ** -14
