"""mla_key_weight where a tile's rows take more than a second: its waits last as long as the work does."""
import pytest
import torch

import attention_prologue_kv_gb300 as kvr

pytestmark = pytest.mark.gpu


def test_rows_that_take_a_pair_more_than_a_second():
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 9 GB")
    H, D, period, times = 128, 8, 4096, 400   # 210 million rows of 8 + 8 channels, 6.5 ns each: 0.82 million groups
    tiles = torch.cuda.get_device_properties(0).multi_processor_count   # two for each pair of CTAs
    T, K, scale = period * times, tiles * 256, 0.35
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    qn, qr = r(period, H, D), r(period, H, D)
    ckv, k = r(tiles * 2, 128, 1, D), r(tiles * 2, 128, 1, D)
    table = torch.randperm(tiles * 2, generator=g, device="cuda").view(1, -1)
    lse = torch.rand(period, H, generator=g, device="cuda") + 10
    i = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
    weight, status = torch.zeros(1, K, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    kvr.mla_key_weight(qn.repeat(times, 1, 1), qr.repeat(times, 1, 1), ckv, k, table, i([0, T]), i([K]), lse.repeat(times, 1), weight,
                       softmax_scale=scale, causal=False, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    # Some keys of each tile. Two halves of the groups' sums are added one after the other in float32: 0.41 million additions, each
    # off by 2^-24 of the whole at most, 2^-5.3 in all; a tile that was cut short lacks far more.
    at = torch.arange(0, K, 257, device="cuda")
    rows = lambda x: x.view(-1, D)[table[0][at // 128] * 128 + at % 128].double()  # noqa: E731
    scores = qn.view(-1, D).double() @ rows(ckv).T + qr.view(-1, D).double() @ rows(k).T
    want = (scale * scores - lse.view(-1, 1).double()).exp_().sum(0) * times
    assert float(((weight[0, at].double() - want) / want).abs().max()) < 2.0 ** -4
