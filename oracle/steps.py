"""A serving step around the paged cache, from its definitions: the batch plan in integers, norms,
rotation, block means and block scores in fp64, the choice of blocks by a plain sort. Test
infrastructure only."""
from __future__ import annotations

import numpy as np

from . import paged as G

OUT_OF_RANGE, SLOT, OUT_OF_PAGES, CAPACITY = 0x1, 0x4, 0x10, 0x20


def _pages(n: int, page: int) -> int:
    return -(-n // page)


def plan(lengths, new, held, table, free, num_free, T, page, seen=None, key_positions=None):
    """The plan's outputs by name, and its error bits; ``table``, ``free`` and ``key_positions`` are changed
    in place. ``seen``: tokens given to each request so far (its length without it)."""
    R, width = table.shape
    err = 0
    lens = [max(int(x), 0) for x in lengths]
    held = [min(max(int(x), 0), width) for x in held]
    top = min(max(int(num_free), 0), len(free))
    goal = [0 if n < 0 else l + int(n) for l, n in zip(lens, new)]
    need = [_pages(g, page) for g in goal]
    for r in range(R):
        for j in range(need[r], held[r]):
            if top < len(free):
                free[top] = table[r, j]
                top += 1
            else:
                err |= SLOT
    have, wanted, tokens = top, 0, 0
    out_len, out_held, cu, req, pos, out_seen, place = [], [], [0], [], [], [], []
    seen = [max(int(x), 0) for x in seen] if seen is not None else lens
    kp_width = 2 ** 31 - 1 if key_positions is None else key_positions.shape[1]
    for r in range(R):
        take, add = max(need[r] - held[r], 0), max(int(new[r]), 0)
        ok = True
        if need[r] > width or max(goal[r], seen[r] + add) > 2 ** 31 - 1 or (add and goal[r] > kp_width):
            err |= OUT_OF_RANGE
            ok = False
        else:
            wanted += take
            tokens += add
            if take and wanted > have:
                err |= OUT_OF_PAGES
                ok = False
            if add and tokens > T:
                err |= CAPACITY
                ok = False
        if ok:
            for j in range(held[r], need[r]):
                top -= 1
                table[r, j] = free[top]
            req += [r] * add
            pos += list(range(lens[r], lens[r] + add))
            place += list(range(seen[r], seen[r] + add))
            if add and key_positions is not None:
                key_positions[r, lens[r]:lens[r] + add] = place[-add:]
        out_seen.append((0 if new[r] < 0 else seen[r] + add) if ok else seen[r])
        out_len.append(goal[r] if ok else lens[r])
        out_held.append(need[r] if ok or need[r] < held[r] else held[r])
        cu.append(len(pos))
    loc = [int(table[r, p // page]) * page + p % page if table[r, p // page] >= 0 else -1 for r, p in zip(req, pos)]
    pad = T - len(pos)
    return {"lengths": out_len, "held": out_held, "num_free": [top], "cu": cu, "req": req + [0] * pad,
            "positions": pos + [-1] * pad, "token_lengths": [p + 1 for p in pos] + [0] * pad,
            "out_loc": loc + [-1] * pad, "seen": out_seen, "token_positions": place + [-1] * pad}, err


def norm_rope(x, n, weight, eps, angles, interleaved):
    """(rows [..., D] after norm and rotation, size [..., D]): ``size`` is |a| + |b| of a rotated
    column's pair, |y| elsewhere. ``angles`` [..., d_rope] of each row, or None."""
    y = np.array(x, dtype=np.float64)
    if n:
        y[..., :n] /= np.sqrt((y[..., :n] ** 2).mean(axis=-1, keepdims=True) + eps)
        if weight is not None:
            y[..., :n] *= weight
    size = np.abs(y)
    if angles is not None:
        half = angles.shape[-1] // 2
        d = y.shape[-1] - 2 * half
        cos, sin = angles[..., :half], angles[..., half:]
        i = np.arange(half)
        ia, ib = (d + 2 * i, d + 2 * i + 1) if interleaved else (d + i, d + half + i)
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def pool(cache, table, page, req, positions, lengths):
    """{page: (mean row, mean of |row|, rows)} of every block that a token lies in."""
    out = {}
    for r, p in zip(req, positions):
        if p < 0:
            continue
        b = int(p) // page
        n = min(int(lengths[r]) - b * page, page)
        slots = int(table[r, b]) * page + np.arange(n)
        rows = G.latent_rows(cache, slots)
        out[int(table[r, b])] = (rows.mean(axis=0), np.abs(rows).mean(axis=0), n)
    return out


def scores(q, summary, pages, scale, weights):
    """(score [n], sum of |w| scale |q||s| [n], sum of |w| relu [n]) of one token over blocks on ``pages``."""
    s = summary[pages]
    x = np.maximum((q @ s.T) * scale, 0.0)
    size = (np.abs(q) @ np.abs(s).T) * scale
    w = np.ones(len(q)) if weights is None else weights
    return w @ x, np.abs(w) @ size, np.abs(w) @ x


def select(row, n_blocks, K, sink, recent):
    """The chosen blocks of one token in ascending order."""
    always = [b for b in range(n_blocks) if b < sink or b >= n_blocks - recent]
    rest = sorted((b for b in range(n_blocks) if b not in set(always)), key=lambda b: (-float(row[b]), b))
    return sorted((always + rest)[:min(K, n_blocks)])
