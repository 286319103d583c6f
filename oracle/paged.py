"""Dense attention over the paged latent cache, attention mass and eviction, in fp64 (numpy), from
their definitions. Test infrastructure only."""
from __future__ import annotations

import numpy as np

from . import projection as P


def _e4m3_values() -> np.ndarray:
    """The 256 e4m3 values: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (c & 0x7F) == 0x7F else (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
        v[c] = -x if c & 0x80 else x
    return v


E4M3 = _e4m3_values()


def latent_rows(cache: np.ndarray, slots) -> np.ndarray:
    """fp64 [n, 256]: bf16 rows (uint16 bits), or packed rows (uint8, 264 bytes) as code * scale."""
    rows = cache[np.asarray(slots, dtype=np.int64)]
    if cache.dtype == np.uint16:
        return P.bf16_to_f64(rows)
    scale = np.ascontiguousarray(rows[:, 256:264]).view(np.float32).astype(np.float64)
    return (E4M3[rows[:, :256]].reshape(-1, 2, 128) * scale[:, :, None]).reshape(-1, 256)


def slots_of(block_table, page_size, num_slots, r, pos):
    """Slots of request r's positions, -1 for one that addresses none."""
    pos = np.asarray(pos, dtype=np.int64)
    if block_table is None:
        return np.where(pos < num_slots, pos, -1)
    page = np.full(pos.shape, -1, dtype=np.int64)
    ok = pos < block_table.shape[1] * page_size
    page[ok] = block_table[r][pos[ok] // page_size]
    slot = page * page_size + pos % page_size
    return np.where((page >= 0) & (slot < num_slots), slot, -1)


def scores(q, cache, block_table, page_size, r, a, b, sm_scale, cap=0.0, slopes=None, qpos=None, kpos=None):
    """(u [H, n], keys [n, 256], pos [n], dot bound [H]) of the valid positions of [a, b); the bound
    is max_j |sm_scale| sum_d |q_d k_jd|."""
    pos = np.arange(max(a, 0), max(b, 0, a))
    if kpos is not None:
        pos = pos[pos < kpos.shape[1]]
    slot = slots_of(block_table, page_size, cache.shape[0], r, pos)
    pos, slot = pos[slot >= 0], slot[slot >= 0]
    k = latent_rows(cache, slot)
    u = (q @ k.T) * sm_scale
    bound = (np.abs(q) @ np.abs(k).T).max(axis=1) * abs(sm_scale) if len(pos) else np.zeros(len(q))
    if cap > 0:
        u = cap * np.tanh(u / cap)
    if slopes is not None:
        kp = pos if kpos is None else kpos[r][pos]
        u = u - np.asarray(slopes, dtype=np.float64)[:, None] * np.abs(float(qpos) - kp)[None, :]
    return u, k, pos, bound


def softmax_output(u, k):
    """(out, lse, sum_j p|k|, sqrt(sum_j (p k)^2)) of one token."""
    if u.shape[1] == 0:
        z = np.zeros((u.shape[0], 256))
        return z, np.full(u.shape[0], -np.inf), z, z
    top = u.max(axis=1, keepdims=True)
    e = np.exp(u - top)
    s = e.sum(axis=1, keepdims=True)
    p = e / s
    return p @ k, (top + np.log(s))[:, 0], p @ np.abs(k), np.sqrt((p * p) @ (k * k))


def evict(lengths, budgets, mass, positions, sink, recent):
    """Per request (length, [(src, dst)], mass row, positions row) after an eviction."""
    out = []
    for r, n in enumerate(lengths):
        n, b = max(int(n), 0), max(int(budgets[r]), 0)
        pos = np.arange(mass.shape[1], dtype=np.int32) if positions is None else positions[r]
        m_row, p_row, moves = mass[r].copy(), pos.copy(), []
        if n > b:
            newest = int(pos[:n].max())
            rank = [np.inf if (pos[j] < sink or pos[j] > newest - recent) else float(mass[r, j]) for j in range(n)]
            kept = set(sorted(range(n), key=lambda j: (-rank[j], j))[:b])
            holes = [j for j in range(b) if j not in kept]
            movers = [j for j in range(b, n) if j in kept]
            moves = list(zip(movers, holes))
            assert len(holes) == len(movers)
            for s, d in moves:
                m_row[d], p_row[d] = mass[r, s], pos[s]
            m_row[b:n] = 0.0
        out.append((min(n, b) if n > b else int(lengths[r]), moves, m_row, p_row))
    return out
