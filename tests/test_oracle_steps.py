"""Pins of oracle/steps.py: closed forms and invariants of the plan, the norms, the block means,
scores and choice."""
import numpy as np

from oracle import steps as S


def test_plan_closed_forms():
    table = np.full((3, 4), -1, dtype=np.int64)
    table[0, :2], table[1, :1] = [7, 3], [5]
    free = np.array([9, 8, 2, -1, -1], dtype=np.int64)
    # request 0 ends, request 1 grows over a page border, request 2 starts
    out, err = S.plan([100, 60, 0], [-1, 10, 65], [2, 1, 0], table, free, 3, 80, 64)
    assert err == 0
    assert out["lengths"] == [0, 70, 65] and out["held"] == [0, 2, 2]
    # 7 and 3 go back; request 1 takes 3, request 2 takes 7 and then 2
    assert table[1].tolist() == [5, 3, -1, -1] and table[2].tolist() == [7, 2, -1, -1] and out["num_free"] == [2]
    assert out["cu"] == [0, 0, 10, 75]
    assert out["positions"][:10] == list(range(60, 70)) and out["req"][10:75] == [2] * 65
    assert out["out_loc"][:10] == [5 * 64 + 60 + i for i in range(4)] + [3 * 64 + i for i in range(6)]
    assert out["out_loc"][74:76] == [2 * 64, -1] and out["token_lengths"][74:76] == [65, 0]


def test_plan_keeps_every_page_once():
    rng = np.random.default_rng(0)
    page, R, width, pages = 16, 20, 12, 150
    table = np.full((R, width), -1, dtype=np.int64)
    free = rng.permutation(pages).astype(np.int64)
    lens, held, top = [0] * R, [0] * R, pages
    for step in range(40):
        new = rng.integers(-1, 30, R)
        out, err = S.plan(lens, new, held, table, free, top, 400, page)
        lens, held, top = out["lengths"], out["held"], out["num_free"][0]
        live = [int(p) for r in range(R) for p in table[r, :held[r]]] + [int(p) for p in free[:top]]
        assert sorted(live) == list(range(pages))
        assert all(h >= -(-n // page) for n, h in zip(lens, held))


def test_norm_and_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 576))
    angle = rng.uniform(0, 6, (5, 32))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    for inter in (False, True):
        y, _ = S.norm_rope(x, 0, None, 1e-6, cs, inter)
        assert np.allclose((y ** 2).sum(axis=1), (x ** 2).sum(axis=1)) and np.array_equal(y[:, :512], x[:, :512])
        back, _ = S.norm_rope(y, 0, None, 1e-6, np.concatenate([np.cos(angle), -np.sin(angle)], axis=1), inter)
        assert np.allclose(back, x)
    for n in (512, 576):
        y, _ = S.norm_rope(x, n, None, 1e-12, None, False)
        assert np.allclose((y[:, :n] ** 2).mean(axis=1), 1.0) and np.array_equal(y[:, n:], x[:, n:])


def test_scores_and_select():
    rng = np.random.default_rng(2)
    q, s = rng.standard_normal((8, 256)), rng.standard_normal((10, 256))
    got, _, _ = S.scores(q, s, [3, 1], 0.5, None)
    want = [sum(max(0.0, 0.5 * float(q[h] @ s[b])) for h in range(8)) for b in (3, 1)]
    assert np.allclose(got, want)
    assert S.select([5, 1, 5, 3, 9], 5, 3, 1, 1) == [0, 2, 4]
    assert S.select([1, 2, 2, 2, 0], 5, 2, 0, 0) == [1, 2]
    assert S.select([0, 0, 0], 2, 5, 1, 1) == [0, 1]
    assert S.select([np.inf, 7, np.inf, 0], 4, 2, 0, 2) == [2, 3]


def test_pool_of_equal_rows():
    cache = np.full((32, 256), 0x3F80, dtype=np.uint16)  # ones
    out = S.pool(cache, np.array([[1, 0]]), 16, [0, 0], [3, 20], [21])
    assert set(out) == {0, 1} and out[0][2] == 5 and out[1][2] == 16
    assert (out[0][0] == 1).all() and (out[1][0] == 1).all()
