"""mla_key_weight: a row whose lse is -inf adds nothing, whatever its query holds (padding of a batch)."""
import numpy as np
import pytest
import torch

from attention_helpers import mla_case
from cache_helpers import check_weight, oracle_weight, row_lse, run_weight

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
FORMS = [dict(H=16, block_size=64), dict(H=128, block_size=64), dict(H=40, block_size=64, dtype="f16"),
         dict(H=16, block_size=100), dict(H=16, block_size=64, k_cache="int8"),
         dict(H=40, block_size=64, cache="int8"), dict(H=16, block_size=64, cache="fp8_e4m3fn", scale_len=512, dtype="f16"),
         dict(H=16, block_size=16, cache="fp8_e5m2", k_cache="fp8_e4m3fn"), dict(H=16, block_size=64, pad=8),
         dict(H=3, block_size=16, Dv=70, Dk=6)]


def poison(c, rows):
    """Queries that a program never filled: NaN, infinities, and products of both signs that overflow."""
    for i, (t, h) in enumerate(rows):
        c.q_nope[t, h] = (NAN, INF, -INF, 1.0)[i % 4]
        c.q_rope[t, h] = (1.0, NAN, INF, -INF)[i % 4]


@pytest.mark.parametrize("kw", FORMS)
@pytest.mark.parametrize("causal", [True, False])
def test_rows_of_a_group(kw, causal):
    """Single rows, all heads of a token, a sequence's first and last row, with finite ones of its group between them."""
    c = mla_case([9, 1, 20], [300, 513, 90], seed=31, causal=causal, **kw)
    H = c.q_nope.shape[1]
    lse = row_lse(c)
    rows = [(0, 0), (3, H - 1), (9, 1 % H), (29, H - 1)] + [(5, h) for h in range(H)] + [(20, h) for h in range(0, H, 2)]
    for t, h in rows:
        lse[t, h] = -np.inf
    width = int(c.key_length.max()) + 3
    past = torch.rand(3, width, generator=torch.Generator().manual_seed(1))
    for old in (None, past):
        want = run_weight(c, lse, width, past=old, decay=0.5)
        check_weight(c, want, oracle_weight(c, lse, width, past=old, decay=0.5), old, 0.5)
    poison(c, rows)
    got = run_weight(c, lse, width, past=past, decay=0.5)
    assert np.array_equal(got[0], want[0]) and got[1] == 0
    check_weight(c, got, oracle_weight(c, lse, width, past=past, decay=0.5), past, 0.5)


@pytest.mark.parametrize("kw", FORMS)
def test_padded_sequences(kw):
    """Sequences all of whose rows are left out, and whole groups of them behind the tokens that count."""
    c = mla_case([4, 70, 1], [300, 700, 40], seed=32, **kw)
    H = c.q_nope.shape[1]
    lse = row_lse(c)
    rows = [(t, h) for t in list(range(4)) + list(range(30, 74)) for h in range(H)]
    for t, h in rows:
        lse[t, h] = -np.inf
    poison(c, rows)
    width = int(c.key_length.max())
    got = run_weight(c, lse, width)
    check_weight(c, got, oracle_weight(c, lse, width))
    # token 25 is the last one that counts: it sees 700 - 70 + 26 keys
    assert (got[0][0, :300] == 0).all() and (got[0][1, :656] > 0).all() and (got[0][1, 656:700] == 0).all()
