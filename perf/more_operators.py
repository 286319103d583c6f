"""Measured cases of the operators around the paged latent cache that make a serving step: the
batch plan (dsa_batch_plan: block tables and slot maps from request lengths), the norms of
queries and keys with the position rotation and the cache write (dsa_qk_norm_rope), and the three
steps that pick the blocks a token attends to (dsa_block_pool: a mean row per block,
dsa_block_scores: a cheap score per token and block, dsa_block_select: the best blocks as a block
table of the token's own, which dsa_paged_attn reads).

``own`` False computes them with elementary torch operations in fp32; ``own`` True calls the
library. Requests hold ragged lengths in pages scattered over one pool, as a serving engine has.
"""
import math

import torch

own = False

DEV = "cuda"
D = 256
EPS = 1e-6
THETA = 10000.0


def listed():
    return [
        # a decode step of a large batch: one token each, some requests end, some were just evicted
        {"name": "plan_decode", "op": "plan", "R": 256, "L": 32768, "new": 1, "page": 64, "end": 16, "evict": 16},
        # prompts arrive: ragged, small pages, each token's slot in one pass
        {"name": "plan_prefill", "op": "plan", "R": 48, "L": 64, "new": 8192, "page": 16, "end": 0, "evict": 0},
        # one token of one request, tensor parallel by four, rotated tail, packed cache: latency is all
        {"name": "norm_one_rope_fp8", "op": "norm", "kind": "fp8", "T": 1, "H": 16, "rope": 64, "inter": 1, "whole": 0},
        # a decode batch without rotation, packed cache
        {"name": "norm_decode_fp8", "op": "norm", "kind": "fp8", "T": 256, "H": 64, "rope": 0, "inter": 0, "whole": 1},
        # a prefill chunk with the rotated tail, bf16 cache
        {"name": "norm_prefill_rope_bf16", "op": "norm", "kind": "bf16", "T": 8192, "H": 64, "rope": 64, "inter": 0,
         "whole": 0},
        # the decode batch's newest block of each request, summed anew
        {"name": "pool_decode_fp8", "op": "pool", "kind": "fp8", "R": 256, "L": 8192, "new": 1, "page": 64},
        # every block of freshly written prompts
        {"name": "pool_prefill_bf16", "op": "pool", "kind": "bf16", "R": 16, "L": 8192, "new": 8192, "page": 64},
        # a few tokens, few heads, small pages, learned head weights: the smallest step
        {"name": "scores_small", "op": "scores", "R": 3, "C": 1, "H": 8, "L": 5000, "page": 16, "w": 1},
        # the decode workload: 256 requests of up to 32768 positions
        {"name": "scores_decode", "op": "scores", "R": 256, "C": 1, "H": 64, "L": 32768, "page": 64, "w": 0},
        # prefill chunks deep in two long documents: a matrix product
        {"name": "scores_prefill", "op": "scores", "R": 2, "C": 2048, "H": 64, "L": 131072, "page": 64, "w": 1},
        # a decode batch over long caches
        {"name": "select_decode", "op": "select", "R": 256, "C": 1, "L": 131072, "page": 64, "K": 64, "sink": 1,
         "recent": 2},
        # a prefill chunk, causal
        {"name": "select_prefill", "op": "select", "R": 4, "C": 2048, "L": 32768, "page": 64, "K": 32, "sink": 1,
         "recent": 2},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "norm", "pool", "scores", "scores", "select"])
    page = rng.choice([1, 16, 33, 48, 64, 64, 128])
    if op == "plan":
        R = _log_int(rng, 1, 1024)
        return {"op": op, "R": R, "L": _log_int(rng, 1, min(131072, 2000000 // R)),
                "new": rng.choice([1, 1, 2, _log_int(rng, 1, min(8192, max(1, 200000 // R)))]),
                "page": page, "end": rng.choice([0, 3, 16]), "evict": rng.choice([0, 5, 16])}
    if op == "norm":
        T = _log_int(rng, 1, 8192)
        return {"op": op, "kind": rng.choice(["bf16", "fp8"]), "T": T, "H": rng.choice([1, 5, 8, 16, 32, 64]),
                "rope": rng.choice([0, 64]), "inter": rng.choice([0, 1]), "whole": rng.choice([0, 1])}
    if op == "pool":
        R = _log_int(rng, 1, 256)
        L = _log_int(rng, 1, min(32768, 131072 // R))
        return {"op": op, "kind": rng.choice(["bf16", "fp8"]), "R": R, "L": L,
                "new": rng.choice([1, 1, _log_int(rng, 1, L), L]), "page": page}
    page = max(page, 16)
    if op == "scores":
        R, C = rng.choice([(_log_int(rng, 1, 256), 1), (_log_int(rng, 1, 8), _log_int(rng, 2, 512))])
        H = rng.choice([1, 5, 8, 16, 32, 48, 64, 64, 128])
        # at most the largest listed case's products, and the decode batch's rows
        L = min(131072, 8000000 // R, page * (536000000 // (R * C * H)))
        return {"op": op, "R": R, "C": C, "H": H, "L": max(C, _log_int(rng, 1, L)), "page": page,
                "w": rng.choice([0, 1])}
    R, C = rng.choice([(_log_int(rng, 1, 256), 1), (_log_int(rng, 1, 8), _log_int(rng, 2, 1024))])
    K = _log_int(rng, 1, 256)
    sink = rng.randint(0, min(K, 2))
    return {"op": op, "R": R, "C": C, "L": max(C, _log_int(rng, 1, min(131072, page * (4000000 // (R * C))))),
            "page": page, "K": K, "sink": sink, "recent": rng.randint(0, min(K - sink, 2))}


# ------------------------------------------------------------------------------- what a case holds --
def _spread(lo, hi, count, salt=0):
    """A fixed spread of host values over [lo, hi], the first one hi."""
    return [hi - ((hi - lo) * (((i + salt * (i > 0)) * 40503) % 65536)) // 65536 for i in range(count)]


def _ceil(a, b):
    return -(-a // b)


def _plan_lists(case):
    """Host lists (length, new tokens, pages held) of a plan's requests."""
    R, page = case["R"], case["page"]
    lens = _spread(max(1, case["L"] // 64), case["L"], R)
    new = _spread(1, case["new"], R, 7)
    held = [_ceil(n, page) for n in lens]
    for i in range(R):
        if case["end"] and i % case["end"] == 2:
            new[i] = -1
        elif case["evict"] and i % case["evict"] == 4:
            lens[i] = _ceil(lens[i], 2)  # the eviction kept half, its pages are not given back yet
    return lens, new, held


def _plan_counts(case):
    """(tokens, pages given back, pages taken) of a plan."""
    lens, new, held = _plan_lists(case)
    need = [_ceil(n + m, case["page"]) if m >= 0 else 0 for n, m in zip(lens, new)]
    return (sum(m for m in new if m > 0), sum(max(0, h - n) for n, h in zip(need, held)),
            sum(max(0, n - h) for n, h in zip(need, held)))


def _pool_lists(case):
    """Host lists (length, new tokens) of a pool's requests."""
    lens = _spread(max(1, case["L"] // 2), case["L"], case["R"])
    return lens, [min(n, case["new"]) for n in lens]


def _lens(case):
    """Host lengths of the requests whose last C tokens ask."""
    return _spread(max(case["C"], case["L"] // 8), case["L"], case["R"])


def _token_lens(case):
    return [n - case["C"] + c + 1 for n in _lens(case) for c in range(case["C"])]


def _table(gen, counts, width):
    """A block table whose pages lie in random order in their pool, and the pool's pages."""
    total = sum(counts) + 8
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    n = torch.tensor(counts, device=DEV)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < n[:, None]] = perm[:sum(counts)]
    return table, total, perm


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _rows(gen, n):
    """Latent rows of unit scale whose magnitude varies from row to row."""
    x = torch.randn((n, D), generator=gen, device=DEV)
    return (x * torch.exp(0.25 * torch.randn((n, 1), generator=gen, device=DEV))).to(torch.bfloat16)


def _cache(gen, kind, slots):
    if kind == "bf16":
        cache = torch.empty((slots, D), dtype=torch.bfloat16, device=DEV)
    else:
        cache = torch.empty((slots, D + 8), dtype=torch.uint8, device=DEV)
    step = 1 << 19
    for s in range(0, slots, step):
        x = _rows(gen, min(step, slots - s))
        if kind == "bf16":
            cache[s:s + step] = x
        else:
            _pack(x.float(), cache[s:s + step], D)
    return cache


def _pack(x, rows, nope):
    """Packed rows of x [n, nope + rope] fp32: e4m3 codes, a scale per 128 columns, a bf16 tail."""
    n, tiles = x.shape[0], nope // 128
    t = x[:, :nope].reshape(n, tiles, 128)
    scale = t.abs().amax(dim=2) / 448.0
    code = torch.where(scale[:, :, None] > 0, t / scale[:, :, None], torch.zeros_like(t))
    rows[:, :nope] = code.to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, nope)
    rows[:, nope:nope + 4 * tiles] = scale.contiguous().view(torch.uint8)
    if x.shape[1] > nope:
        rows[:, nope + 4 * tiles:] = x[:, nope:].to(torch.bfloat16).contiguous().view(torch.uint8)


def _cache_views(case, cache):
    """What a cache holds, as values: rows, or codes, scales and the tail."""
    if case["kind"] == "bf16":
        return {"cache": cache}
    nope = 512 if case["rope"] else 256
    got = {"codes": cache[:, :nope].view(torch.float8_e4m3fn),
           "scales": cache[:, nope:nope + nope // 32].view(torch.float32)}
    if case["rope"]:
        got["tail"] = cache[:, nope + nope // 32:].view(torch.bfloat16)
    return got


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, page = case["op"], case.get("page")
    if op == "plan":
        lens, new, held = _plan_lists(case)
        tokens, back, taken = _plan_counts(case)
        width = max(max(held), max(_ceil(n + max(m, 0), page) for n, m in zip(lens, new))) + 1
        table, total, perm = _table(gen, held, width)
        spare = taken + 64
        free = torch.full((total + spare,), -1, dtype=torch.int32, device=DEV)
        free[:spare + 8] = torch.cat([perm[sum(held):], total + torch.randperm(spare, generator=gen, device=DEV).to(torch.int32)])
        T = _ceil(tokens, 64) * 64  # a captured step has room to spare
        i32 = {"dtype": torch.int32, "device": DEV}
        return {"case": case, "lengths": _i32(lens), "new": _i32(new), "held": _i32(held), "table": table, "free": free,
                "num_free": _i32([spare + 8]), "T": T, "tokens": tokens, "back": back, "taken": taken,
                "out": {"lengths": torch.zeros(case["R"], **i32), "held": torch.zeros(case["R"], **i32),
                        "num_free": torch.zeros(1, **i32)}}
    if op == "norm":
        T, H, rope = case["T"], case["H"], case["rope"]
        nope = 512 if rope else 256
        dim = nope + rope
        slots = T + T // 4 + 8
        x = {"case": case, "q": torch.randn((T, H, dim), generator=gen, device=DEV, dtype=torch.bfloat16)}
        x["q"] *= torch.exp(0.5 * torch.randn((T, H, 1), generator=gen, device=DEV)).to(torch.bfloat16)
        x["k"] = (3.0 * torch.randn((T, dim), generator=gen, device=DEV)).to(torch.bfloat16)
        x["n"] = dim if case["whole"] else nope
        x["q_weight"] = (1 + 0.1 * torch.randn(x["n"], generator=gen, device=DEV)).to(torch.bfloat16)
        x["k_weight"] = (1 + 0.1 * torch.randn(x["n"], generator=gen, device=DEV)).to(torch.bfloat16)
        x["positions"] = torch.randint(0, 16384, (T,), generator=gen, device=DEV).to(torch.int32)
        x["out_loc"] = torch.randperm(slots, generator=gen, device=DEV)[:T]
        x["cos_sin"] = None
        if rope:
            at = torch.arange(16384, device=DEV, dtype=torch.float64)
            angle = at[:, None] * THETA ** (-2.0 * torch.arange(rope // 2, device=DEV, dtype=torch.float64) / rope)
            x["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        x["q_out"] = torch.zeros_like(x["q"])
        if case["kind"] == "bf16":
            x["cache"] = torch.zeros((slots, dim), dtype=torch.bfloat16, device=DEV)
        else:
            x["cache"] = torch.zeros((slots, nope + nope // 32 + 2 * rope), dtype=torch.uint8, device=DEV)
        return x
    if op == "pool":
        lens, new = _pool_lists(case)
        counts = [_ceil(n, page) for n in lens]
        table, total, _ = _table(gen, counts, max(counts) + 1)
        req = [r for r, m in enumerate(new) for _ in range(m)]
        pos = [n - m + i for n, m in zip(lens, new) for i in range(m)]
        blocks = sum(c - (n - m) // page for c, n, m in zip(counts, lens, new))
        return {"case": case, "cache": _cache(gen, case["kind"], total * page), "table": table, "lengths": _i32(lens),
                "new": _i32(new), "req": _i32(req), "positions": _i32(pos), "blocks": blocks,
                "summary": torch.zeros((total, D), dtype=torch.bfloat16, device=DEV)}
    lens, tlens = _lens(case), _i32(_token_lens(case))
    counts = [_ceil(n, page) for n in lens]
    width = max(counts) + 1
    table, total, _ = _table(gen, counts, width)
    T = case["R"] * case["C"]
    state = {"case": case, "table": table, "lengths": tlens, "width": width,
             "req": torch.arange(T, device=DEV, dtype=torch.int32) // case["C"]}
    if op == "scores":
        state["q"] = torch.randn((T, case["H"], D), generator=gen, device=DEV).to(torch.bfloat16)
        # means of a page's rows: their spread shrinks with the page, but neighbours share a direction
        state["summary"] = (torch.randn((total, D), generator=gen, device=DEV) / math.sqrt(page) + 0.05).to(torch.bfloat16)
        state["weights"] = (torch.rand((T, case["H"]), generator=gen, device=DEV) - 0.1) if case["w"] else None
        state["scores"] = torch.zeros((T, width), device=DEV)
        return state
    state["scores"] = torch.exp(torch.randn((T, width), generator=gen, device=DEV))
    # blocks that no head looks at: equal scores of zero
    state["scores"][torch.rand((T, width), generator=gen, device=DEV) < 0.05] = 0.0
    return state


# ------------------------------------------------------------------------------------- the passes --
def _run_own(state):
    import dsa_sparse_attention_mla_gb300 as dsa

    case = state["case"]
    op = case["op"]
    if op == "plan":
        out = state["out"]
        cu, req, pos, tlen, loc = dsa.dsa_batch_plan(
            state["lengths"], state["new"], state["held"], state["table"], state["free"], state["num_free"], state["T"],
            page_size=case["page"], lengths_out=out["lengths"], held_out=out["held"], num_free_out=out["num_free"])
        return {**out, "cu": cu, "req": req, "positions": pos, "token_lengths": tlen, "out_loc": loc,
                "table": state["table"], "free": state["free"]}
    if op == "norm":
        kind = dsa.CACHE_FP8_SCALED if case["kind"] == "fp8" else dsa.CACHE_BF16
        rope = case["rope"]
        dsa.dsa_qk_norm_rope(state["q"], state["k"], state["positions"], state["cos_sin"], EPS, state["cache"], kind,
                             state["out_loc"], d_nope=512 if rope else 256, d_rope=rope, q_norm=state["n"],
                             k_norm=state["n"], q_weight=state["q_weight"], k_weight=state["k_weight"],
                             interleaved=bool(case["inter"]), q_out=state["q_out"])
        return {"q": state["q_out"], **_cache_views(case, state["cache"])}
    if op == "pool":
        kind = dsa.CACHE_FP8_SCALED if case["kind"] == "fp8" else dsa.CACHE_BF16
        dsa.dsa_block_pool(state["cache"], kind, state["table"], state["positions"], state["lengths"], state["summary"],
                           page_size=case["page"], req_of_token=state["req"])
        return {"summary": state["summary"]}
    if op == "scores":
        dsa.dsa_block_scores(state["q"], state["summary"], state["table"], state["lengths"], 1.0 / 16.0,
                             page_size=case["page"], req_of_token=state["req"], weights=state["weights"],
                             out=state["scores"])
        return {"scores": state["scores"]}
    blocks, table, lengths = dsa.dsa_block_select(state["scores"], state["table"], state["lengths"], case["K"],
                                                  page_size=case["page"], req_of_token=state["req"], sink=case["sink"],
                                                  recent=case["recent"])
    return {"blocks": blocks, "table": table, "lengths": lengths}


def _run_plan(state):
    page, T, table, free = state["case"]["page"], state["T"], state["table"], state["free"]
    R, width = table.shape
    n, h, nf = state["lengths"].long().clamp(min=0), state["held"].long(), state["num_free"].long()
    add = state["new"].long()
    after = torch.where(add < 0, torch.zeros_like(n), n + add.clamp(min=0))
    need = (after + page - 1) // page
    fits = need <= width
    back = (h - need).clamp(min=0)
    take = torch.where(fits, (need - h).clamp(min=0), torch.zeros_like(h))
    tok = torch.where(fits, add.clamp(min=0), torch.zeros_like(h))
    have = nf + back.sum()
    ok = fits & ((take == 0) | (take.cumsum(0) <= have)) & ((tok == 0) | (tok.cumsum(0) <= T))
    take, tok = take * ok, tok * ok
    # pages given back go on top of the free ones, in the order of requests and pages
    r = torch.arange(R, device=DEV)
    who = torch.repeat_interleave(r, back, output_size=state["back"])
    i = torch.arange(state["back"], device=DEV)
    free[nf + i] = table[who, need[who] + i - (back.cumsum(0) - back)[who]]
    # pages taken come from the top
    who = torch.repeat_interleave(r, take, output_size=state["taken"])
    i = torch.arange(state["taken"], device=DEV)
    table[who, h[who] + i - (take.cumsum(0) - take)[who]] = free[have - 1 - i]
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), tok.cumsum(0)])
    i = torch.arange(T, device=DEV)
    live = i < cu[-1]
    who = torch.searchsorted(cu[1:], i, right=True).clamp(max=R - 1)
    pos = n[who] + i - cu[who]
    slot = table[who, torch.where(live, pos, 0) // page].long() * page + pos % page
    i32 = torch.int32
    out = state["out"]
    out["lengths"].copy_(torch.where(ok, after, n))
    out["held"].copy_(torch.where(ok & (take > 0), need, torch.minimum(h, need)))
    out["num_free"].copy_(have - take.sum())
    return {**out, "cu": cu.to(i32), "req": torch.where(live, who, 0).to(i32),
            "positions": torch.where(live, pos, -1).to(i32), "token_lengths": torch.where(live, pos + 1, 0).to(i32),
            "out_loc": torch.where(live, slot, -1), "table": table, "free": free}


def _normed(x, n, weight, cos_sin, positions, rope, interleaved):
    """x [T, H, dim] in fp32: the norm of the first n columns, then the rotation of the last ones."""
    x = x.float()
    head = x[..., :n]
    head = head * torch.rsqrt((head * head).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    x = torch.cat([head, x[..., n:]], dim=-1)
    if rope == 0:
        return x
    t = x[..., -rope:]
    angle = cos_sin[positions.long()][:, None, :]
    cos, sin = angle[..., :rope // 2], angle[..., rope // 2:]
    a, b = (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., :rope // 2], t[..., rope // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    t = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([x[..., :-rope], t], dim=-1)


def _run_norm(state):
    case = state["case"]
    rope, args = case["rope"], (state["cos_sin"], state["positions"], case["rope"], case["inter"])
    state["q_out"].copy_(_normed(state["q"], state["n"], state["q_weight"], *args))
    k = _normed(state["k"][:, None, :], state["n"], state["k_weight"], *args)[:, 0]
    if case["kind"] == "bf16":
        state["cache"][state["out_loc"]] = k.to(torch.bfloat16)
    else:
        rows = torch.empty((case["T"], state["cache"].shape[1]), dtype=torch.uint8, device=DEV)
        _pack(k, rows, 512 if rope else 256)
        state["cache"][state["out_loc"]] = rows
    return {"q": state["q_out"], **_cache_views(case, state["cache"])}


def _run_pool(state):
    case, page = state["case"], state["case"]["page"]
    n = state["lengths"].long()
    first = (n - state["new"]) // page
    count = (n + page - 1) // page - first
    who = torch.repeat_interleave(torch.arange(case["R"], device=DEV), count, output_size=state["blocks"])
    block = first[who] + torch.arange(state["blocks"], device=DEV) - (count.cumsum(0) - count)[who]
    where = state["table"][who, block].long()
    raw = state["cache"].view(-1, page, state["cache"].shape[1])[where]
    if case["kind"] == "bf16":
        rows = raw.float()
    else:
        code = raw[..., :D].contiguous().view(torch.float8_e4m3fn).float().view(-1, page, 2, 128)
        rows = (code * raw[..., D:].contiguous().view(torch.float32)[..., None]).view(-1, page, D)
    held = (n[who] - block * page).clamp(max=page)
    live = torch.arange(page, device=DEV)[None, :] < held[:, None]
    total = torch.where(live[:, :, None], rows, torch.zeros_like(rows)).sum(dim=1)
    state["summary"][where] = (total / held[:, None]).to(torch.bfloat16)
    return {"summary": state["summary"]}


def _run_scores(state):
    case = state["case"]
    R, C, H, width = case["R"], case["C"], case["H"], state["width"]
    rows = state["summary"][state["table"].clamp(min=0).long()].float()  # [R, width, 256]
    x = torch.bmm(state["q"].float().view(R, C * H, D), rows.transpose(1, 2)).view(R * C, H, width)
    x = torch.clamp(x * (1.0 / 16.0), min=0)
    if state["weights"] is not None:
        x = x * state["weights"][:, :, None]
    blocks = (state["lengths"] + case["page"] - 1) // case["page"]
    live = torch.arange(width, device=DEV)[None, :] < blocks[:, None]
    state["scores"].copy_(torch.where(live, x.sum(dim=1), state["scores"]))
    return {"scores": state["scores"]}


def _run_select(state):
    case, K, page = state["case"], state["case"]["K"], state["case"]["page"]
    n, width = state["lengths"].long(), state["width"]
    nb = ((n + page - 1) // page)[:, None]
    b = torch.arange(width, device=DEV)[None, :]
    # 0: outside, 1: by score, 2: always; ordered by score, then, stably, by these
    rank = (b < nb).long() + ((b < nb) & ((b < case["sink"]) | (b >= nb - case["recent"]))).long()
    order = torch.sort(state["scores"], dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(rank.gather(1, order), dim=1, descending=True, stable=True).indices)
    if width < K:
        order = torch.cat([order, order.new_full((order.shape[0], K - width), width)], dim=1)
    kept = torch.arange(K, device=DEV)[None, :] < nb
    picked = torch.sort(torch.where(kept, order[:, :K], width), dim=1).values
    kept = picked < width
    picked = torch.where(kept, picked, 0)
    table = torch.where(kept, state["table"][state["req"].long()[:, None], picked], -1)
    count = kept.sum(dim=1)
    last = (kept & (picked == nb - 1)).any(dim=1)
    lengths = count * page - torch.where(last, nb[:, 0] * page - n, torch.zeros_like(n))
    return {"blocks": torch.where(kept, picked, -1).to(torch.int32), "table": table, "lengths": lengths.to(torch.int32)}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "plan":
        return _run_plan(state)
    if op == "norm":
        return _run_norm(state)
    if op == "pool":
        return _run_pool(state)
    if op == "scores":
        return _run_scores(state)
    return _run_select(state)


def work(case):
    op, page = case["op"], case.get("page")
    if op == "plan":
        tokens, back, taken = _plan_counts(case)
        T = _ceil(tokens, 64) * 64
        # the state in and out, the scan, each page moved read and written, the page a run of tokens
        # lies in, and the tokens' entries
        return {"bytes": case["R"] * 24 + 8 * (back + taken) + 4 * _ceil(tokens, page) + T * 20, "flops": 0}
    if op == "norm":
        T, H, rope = case["T"], case["H"], case["rope"]
        nope = 512 if rope else 256
        dim = nope + rope
        row = 2 * dim if case["kind"] == "bf16" else nope + nope // 32 + 2 * rope
        n = dim if case["whole"] else nope
        return {"bytes": T * (4 * H * dim + 2 * dim + row + 8 + (4 + 4 * rope if rope else 0)) + 4 * n,
                "flops": T * (H + 1) * 4 * dim}
    if op == "pool":
        lens, new = _pool_lists(case)
        row = 512 if case["kind"] == "bf16" else D + 8
        rows = sum(n - (n - m) // page * page for n, m in zip(lens, new))
        blocks = sum(_ceil(n, page) - (n - m) // page for n, m in zip(lens, new))
        return {"bytes": rows * row + blocks * (512 + 4) + 8 * sum(new), "flops": rows * D}
    lens, tlens = _lens(case), _token_lens(case)
    pairs, T = sum(_ceil(n, page) for n in tlens), len(tlens)
    if op == "scores":
        rows = sum(_ceil(n, page) for n in lens)
        return {"bytes": rows * (512 + 4) + T * case["H"] * (512 + 4 * case["w"]) + T * 8 + 4 * pairs,
                "flops": 2 * pairs * case["H"] * D}
    return {"bytes": 4 * pairs + T * (12 + 8 * case["K"]) + 4 * sum(min(case["K"], _ceil(n, page)) for n in tlens),
            "flops": 0}


# ------------------------------------------------------------------- the definitions in 64 bits --
def _exact_plan(st):
    case, T = st["case"], st["T"]
    page = case["page"]
    table, free = st["table"].tolist(), st["free"].tolist()
    top = int(st["num_free"])
    lens, new, held = st["lengths"].tolist(), st["new"].tolist(), st["held"].tolist()
    goal = [0 if m < 0 else n + m for n, m in zip(lens, new)]
    for r, g in enumerate(goal):
        while held[r] > _ceil(g, page) and held[r] > 0:
            free[top:top + held[r] - _ceil(g, page)] = table[r][_ceil(g, page):held[r]]
            top += held[r] - _ceil(g, page)
            held[r] = _ceil(g, page)
    cu, req, pos = [0], [], []
    for r, g in enumerate(goal):
        while held[r] < _ceil(g, page):
            top -= 1
            table[r][held[r]] = free[top]
            held[r] += 1
        fresh = range(lens[r], g) if new[r] > 0 else range(0)
        req += [r] * len(fresh)
        pos += list(fresh)
        cu.append(len(pos))
    pad = T - len(pos)
    loc = [table[r][p // page] * page + p % page for r, p in zip(req, pos)] + [-1] * pad
    return {"lengths": _i32(goal), "held": _i32(held), "num_free": _i32([top]), "cu": _i32(cu), "req": _i32(req + [0] * pad),
            "positions": _i32(pos + [-1] * pad), "token_lengths": _i32([p + 1 for p in pos] + [0] * pad),
            "out_loc": torch.tensor(loc, device=DEV), "table": _i32(table), "free": _i32(free)}


def _exact_rows(st, x, weight):
    """Normalised and rotated rows of x [T, ..., dim] in fp64, the rotation as a complex product."""
    case, n = st["case"], st["n"]
    y = x.to(torch.float64)
    y[..., :n] /= torch.sqrt(torch.einsum("...d,...d->...", y[..., :n], y[..., :n]) / n + EPS)[..., None]
    y[..., :n] *= weight.to(torch.float64)
    if case["rope"]:
        tail = y[..., -64:].clone()
        pairs = tail.unflatten(-1, (32, 2)) if case["inter"] else tail.unflatten(-1, (2, 32)).transpose(-1, -2)
        turn = st["cos_sin"].to(torch.float64)[st["positions"].long()].unflatten(-1, (2, 32)).transpose(-1, -2)
        turn = torch.view_as_complex(turn.contiguous()).view(-1, *[1] * (x.dim() - 2), 32)
        tail = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y[..., -64:] = (tail if case["inter"] else tail.transpose(-1, -2)).flatten(-2)
    return y


def _exact_norm(st):
    case = st["case"]
    nope = 512 if case["rope"] else 256
    k = _exact_rows(st, st["k"], st["k_weight"])
    slots, loc = st["cache"].shape[0], st["out_loc"]

    def placed(rows):
        full = torch.zeros((slots, rows.shape[1]), dtype=torch.float64, device=DEV)
        return full.index_copy_(0, loc, rows)

    got = {"q": _exact_rows(st, st["q"], st["q_weight"])}
    if case["kind"] == "bf16":
        return {**got, "cache": placed(k)}
    tiles = k[:, :nope].unflatten(-1, (nope // 128, 128))
    scale = tiles.abs().amax(dim=-1) / 448
    got.update(codes=placed((tiles / scale[..., None]).flatten(-2)), scales=placed(scale))  # before any rounding
    if case["rope"]:
        got["tail"] = placed(k[:, nope:])
    return got


def _exact_pool(st):
    case, page = st["case"], st["case"]["page"]
    out = torch.zeros(st["summary"].shape, dtype=torch.float64, device=DEV)
    lens, new = _pool_lists(case)
    for r, (n, m) in enumerate(zip(lens, new)):
        a = (n - m) // page * page  # whole blocks from here on
        j = torch.arange(a, n, device=DEV)
        where = st["table"][r].long()[j // page]
        raw = st["cache"].index_select(0, where * page + j % page)
        if case["kind"] == "bf16":
            x = raw.double()
        else:
            x = raw[:, :D].contiguous().view(torch.float8_e4m3fn).float().double()
            x = x * raw[:, D:].contiguous().view(torch.float32).double().repeat_interleave(128, dim=1)
        out.index_add_(0, where, x)
        hits = torch.zeros(out.shape[0], dtype=torch.float64, device=DEV).index_add_(0, where, torch.ones_like(x[:, 0]))
        out /= torch.where(hits > 0, hits, torch.ones_like(hits))[:, None]
    return {"summary": out}


def _exact_scores(st):
    case, C, page = st["case"], st["case"]["C"], st["case"]["page"]
    out = st["scores"].double()
    for r, n in enumerate(_lens(case)):
        p = st["summary"][st["table"][r, :_ceil(n, page)].long()].double()
        for a in range(r * C, (r + 1) * C, 256):
            b = min(a + 256, (r + 1) * C)
            x = torch.einsum("thd,bd->htb", st["q"][a:b].double(), p).clamp_(min=0) / 16
            w = torch.ones((b - a, case["H"]), dtype=torch.float64, device=DEV) if st["weights"] is None else st["weights"][a:b].double()
            s = torch.einsum("htb,th->tb", x, w)
            live = torch.arange(p.shape[0], device=DEV)[None, :] * page < st["lengths"][a:b, None]
            out[a:b, :p.shape[0]][live] = s[live]
    return {"scores": out}


def _exact_select(st):
    import numpy as np

    case, K, page = st["case"], st["case"]["K"], st["case"]["page"]
    scores, table = st["scores"].cpu().numpy().astype(np.float64), st["table"].cpu().numpy()
    T = scores.shape[0]
    blocks, own_table = np.full((T, K), -1, np.int32), np.full((T, K), -1, np.int32)
    lengths = np.zeros(T, np.int32)
    for t, n in enumerate(_token_lens(case)):
        nb = _ceil(n, page)
        s = scores[t, :nb].copy()
        s[:case["sink"]] = np.inf
        s[max(0, nb - case["recent"]):] = np.inf
        best = np.sort(np.lexsort((np.arange(nb), -s))[:K])
        blocks[t, :best.size] = best
        own_table[t, :best.size] = table[t // case["C"], best]
        lengths[t] = np.minimum(page, n - best * page).sum()
    return {"blocks": torch.from_numpy(blocks), "table": torch.from_numpy(own_table), "lengths": torch.from_numpy(lengths)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "norm": _exact_norm, "pool": _exact_pool, "scores": _exact_scores,
            "select": _exact_select}[case["op"]](st)
