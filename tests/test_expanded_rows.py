"""A tensor that is one row expanded has row stride 0, which the C ABI reads as dense rows: the binding refuses it, as
the call would go past the row's storage."""
import pytest
import torch

import attention_prologue_kv_gb300 as kvr
from attention_prologue_kv_gb300.api import _kv_rows

SHAPES = [((1, 24), (3, 24)), ((1, 1, 24), (1, 3, 24)), ((1, 1, 24), (2, 3, 24)), ((1, 1, 1, 24), (1, 1, 3, 24)),
          ((1, 1, 1, 24), (2, 1, 1, 24)), ((1, 1, 1, 24), (2, 1, 3, 24))]


@pytest.mark.parametrize("one,many", SHAPES)
def test_rows_of_an_expanded_tensor(one, many):
    x = torch.zeros(one, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expanded"):
        _kv_rows(x.expand(many))
    dense = torch.zeros(many, dtype=torch.bfloat16)
    assert _kv_rows(dense)[2] == 24 and _kv_rows(x)[:2] == (1, 1)
    assert _kv_rows(torch.zeros(many[:-1] + (40,), dtype=torch.bfloat16)[..., :24])[2] == 40


def test_a_single_row_may_have_any_stride():
    x = torch.zeros(24, dtype=torch.bfloat16)
    assert _kv_rows(x.as_strided((1, 24), (0, 1)))[:2] == (1, 1)
    assert _kv_rows(x.as_strided((0, 24), (0, 1)))[:2] == (0, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("one,many", SHAPES)
def test_calls_refuse_expanded_rows(one, many):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    ckv, k = z(2, 4, 1, 16), z(2, 4, 1, 8)
    rows = torch.Size(many[:-1]).numel()
    index = torch.arange(rows, device="cuda")
    with pytest.raises(ValueError, match="expanded"):
        kvr.kv_cache_read(ckv, k, index, z(*one).expand(many))
    with pytest.raises(ValueError, match="expanded"):
        kvr.kv_rmsnorm_rope_cache(z(*one).expand(many), z(16), z(rows, 8), z(rows, 8), index, ckv, k)
    with pytest.raises(ValueError, match="expanded"):
        kvr.dynamic_quant(z(*one).expand(many), z(*many, dtype=torch.int8), z(rows, dtype=torch.float32))
