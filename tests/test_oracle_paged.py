"""Pins of the fp64 definitions in oracle/paged.py: closed forms and torch's own dense attention."""
import numpy as np
import pytest

from oracle import paged as R
from oracle import projection as P


def test_e4m3_table():
    assert R.E4M3[0x7E] == 448 and R.E4M3[0x01] == 2.0 ** -9 and R.E4M3[0x38] == 1.0 and R.E4M3[0xB8] == -1.0
    assert np.isnan(R.E4M3[0x7F]) and np.isnan(R.E4M3[0xFF])
    fin = [c for c in range(256) if (c & 0x7F) != 0x7F]
    assert np.array_equal(R.E4M3[fin], P.e4m3_decode(np.array(fin, dtype=np.uint8)))


def test_attention_matches_torch():
    import torch

    rng = np.random.default_rng(0)
    cache = P.f64_to_bf16(rng.standard_normal((96, 256)))
    q = rng.standard_normal((4, 256))
    bt = np.array([[2, 0, 1]])
    u, k, pos, _ = R.scores(q, cache, bt, 32, 0, 5, 90, 0.125)
    rows = P.bf16_to_f64(cache)[[bt[0][j // 32] * 32 + j % 32 for j in range(5, 90)]]
    ref = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(x)[None] for x in (q, rows, rows)),
                                                           scale=0.125)
    out, lse, _, _ = R.softmax_output(u, k)
    assert np.allclose(out, ref[0].numpy(), atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(q @ rows.T * 0.125), 1).numpy())


def test_cap_and_bias_closed_forms():
    cache = P.f64_to_bf16(np.ones((4, 256)))
    q = np.full((2, 256), 1.0)
    u, _, _, _ = R.scores(q, cache, None, 1, 0, 0, 4, 1.0, cap=10.0, slopes=np.array([0.0, 2.0]), qpos=3)
    assert np.allclose(u[0], 10.0) and np.allclose(u[1], 10.0 - 2.0 * np.array([3, 2, 1, 0]))


def test_slots_and_masking():
    bt = np.array([[1, -1, 9]])
    assert R.slots_of(bt, 4, 16, 0, [0, 3, 4, 8, 12]).tolist() == [4, 7, -1, -1, -1]
    out, lse, _, _ = R.softmax_output(np.zeros((3, 0)), np.zeros((0, 256)))
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("budget", [0, 1, 3, 5, 6])
def test_evict_small(budget):
    mass = np.array([[5.0, 1.0, 4.0, 1.0, 3.0, 0.0]], dtype=np.float32)
    n, moves, m, p = R.evict([6], [budget], mass, None, 0, 0)[0]
    assert n == min(6, budget)
    want = {0: [], 1: [5.0], 3: [3.0, 4.0, 5.0], 5: [1.0, 1.0, 3.0, 4.0, 5.0], 6: [0.0, 1.0, 1.0, 3.0, 4.0, 5.0]}
    assert sorted(m[:n].tolist()) == want[budget]
    if budget == 3:
        assert moves == [(4, 1)] and p[:3].tolist() == [0, 4, 2] and m[3:].tolist() == [0, 0, 0]
    # protected: the newest stays whatever its mass
    if budget == 1:
        assert R.evict([6], [1], mass, None, 0, 1)[0][1] == [(5, 0)]
