"""Pins of the oracle's attention step: closed forms and library routines."""
import numpy as np
import pytest
import torch

import oracle
from attention_helpers import mla_case, oracle_mla


def test_rope_is_complex_multiplication_per_axis():
    rng = np.random.default_rng(0)
    q = rng.standard_normal((5, 3, 16))
    pos = rng.integers(-50, 10 ** 6, (3, 5))
    sections = [2, 5, 1]
    for half in (False, True):
        out, cos, sin = oracle.ref_query_rope(q, pos, sections, 500.0, half)
        axis = [0, 0, 1, 1, 1, 1, 1, 2]
        for i in range(8):
            turn = pos[axis[i]] * 500.0 ** (-i / 8)
            z = q[..., i] + 1j * q[..., i + 8] if half else q[..., 2 * i] + 1j * q[..., 2 * i + 1]
            w = z * np.exp(1j * turn)[:, None]
            assert np.allclose(out[..., i], w.real, atol=1e-12) and np.allclose(out[..., i + 8], w.imag, atol=1e-12)
            assert np.allclose(cos[:, i], np.cos(turn)) and np.array_equal(cos[:, i], cos[:, i + 8])
            assert np.allclose(sin[:, i + 8], np.sin(turn))


def test_rope_of_one_axis_is_the_prologue_rotation():
    """The tables it writes make the key's interleaved RoPE turn the same way."""
    rng = np.random.default_rng(1)
    q = rng.standard_normal((4, 1, 8))
    out, cos, sin = oracle.ref_query_rope(q, rng.integers(0, 99, (1, 4)), [4])
    assert np.allclose(out[:, 0], oracle.interleave_rope(q[:, 0], cos, sin), atol=1e-13)


def test_read_inverts_the_scatter():
    rng = np.random.default_rng(2)
    index = np.array([7, -1, 0, 12, 3, 99])
    ckv, k = rng.integers(-9, 9, (4, 4, 6)).astype(float), rng.standard_normal((4, 4, 2))
    out = np.full((2, 3, 8), 5.0)
    assert oracle.ref_kv_cache_read(out, ckv, k, index, "PA_BSND", ckv_scale=np.arange(1.0, 7)) == 1
    flat = out.reshape(6, 8)
    assert (flat[1] == 5).all() and (flat[5] == 5).all()
    for t, slot in ((0, 7), (2, 0), (3, 12), (4, 3)):
        assert np.allclose(flat[t, :6] * np.arange(1, 7), ckv.reshape(16, 6)[slot]) and (flat[t, 6:] == k.reshape(16, 2)[slot]).all()


@pytest.mark.parametrize("causal", [True, False])
def test_attention_equals_torch_sdpa(causal):
    """Against scaled_dot_product_attention in float64 on the gathered keys."""
    c = mla_case([3, 1, 5], [9, 33, 5], H=2, Dv=12, Dk=4, block_size=4, causal=causal, seed=3)
    out, lse, st, A, B = oracle_mla(c)
    assert st == 0
    for n in range(3):
        a, b, K = int(c.query_start[n]), int(c.query_start[n + 1]), int(c.key_length[n])
        i = torch.arange(K)
        slot = c.table[n, i // 4] * 4 + i % 4
        v = c.ckv.view(-1, 12)[slot].double()
        key = torch.cat([v, c.k.view(-1, 4)[slot].double()], -1)
        q = torch.cat([c.q_nope, c.q_rope], -1)[a:b].double().transpose(0, 1)
        mask = (i[None] <= (K - (b - a) + torch.arange(b - a))[:, None]) if causal else torch.ones(b - a, K, dtype=torch.bool)
        want = torch.nn.functional.scaled_dot_product_attention(q, key.expand(2, -1, -1), v.expand(2, -1, -1), attn_mask=mask,
                                                                scale=float(np.float32(c.scale)))
        assert np.allclose(out[a:b], want.transpose(0, 1).numpy(), atol=1e-12)
        s = (q @ key.T * float(np.float32(c.scale))).masked_fill(~mask, -torch.inf)
        assert np.allclose(lse[a:b], torch.logsumexp(s, -1).T.numpy(), atol=1e-12)


def test_attention_edges():
    """More new tokens than keys, no keys, a hole over all of them: zeros and
    -inf; left-out sequences and rows behind the last stay."""
    c = mla_case([4, 2, 1, 1], [2, 0, 3, 3], H=1, Dv=4, Dk=2, block_size=4, holes=[(2, 0)], gap=2, seed=4)
    c.key_length[3] = 10 ** 6
    out, lse, st, _, _ = oracle_mla(c)
    assert st == 0x2
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:4]).all()
    assert (out[4:7] == 0).all() and np.isneginf(lse[4:7]).all()
    assert (out[7:] == -77).all() and (lse[7:] == -77).all()
    c.key_length[3] = 3
    c.table[0, 0] = c.ckv.shape[0]
    c.query_start[4] = 99
    assert oracle_mla(c)[2] == 0x21
