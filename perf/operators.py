"""Measured cases of the dense paged latent-cache operators: attention of one new token per
request (dsa_paged_attn), the accumulation of its attention weight per cached position
(dsa_paged_attn_mass) and the eviction of the lightest positions (dsa_cache_evict).

``own`` False computes them with elementary torch operations in fp32; ``own`` True calls the
library. Requests hold ragged lengths in pages scattered over one pool, as a serving engine has.
"""
import math

import torch

own = False

DEV = "cuda"
D = 256
ROW_FP8 = 264

_BASE = {"kind": "fp8", "T": 1, "H": 64, "L": 1024, "Lmin": 1024, "page": 64, "cap": 0.0, "bias": 0, "doc": 0}


def _attn(name, **kw):
    return {"name": name, "op": "attn", **_BASE, **kw}


def _mass(name, **kw):
    return {"name": name, "op": "mass", **_BASE, **kw}


def _evict(name, **kw):
    return {"name": name, "op": "evict", "kind": "fp8", "R": 1, "L": 1024, "Lmin": 1024, "page": 64, "budget": 512,
            "sink": 4, "recent": 64, **kw}


def listed():
    return [
        # the first tokens of a chat: one request, less than one page and a half; latency is all
        _attn("attn_one_short_bf16", kind="bf16", T=1, L=97, Lmin=97),
        # a small batch at the top-k's own length, where a sparse layer gains nothing yet
        _attn("attn_small_batch_fp8", T=8, L=2112, Lmin=1900),
        # an ordinary ragged decode batch on a bf16 cache
        _attn("attn_batch_bf16", kind="bf16", T=64, L=8192, Lmin=300),
        # the decode workload's length per request, every request full: the largest call
        _attn("attn_batch_fp8_32k", T=128, L=32768, Lmin=32768),
        # one long document: the length has to be split over the whole device and joined
        _attn("attn_one_long_fp8", T=1, L=131071, Lmin=131071),
        # capped scores with a distance bias and packed documents (each token sees its own one),
        # half the heads (tensor parallel by two), small pages
        _attn("attn_cap_bias_doc_bf16", kind="bf16", T=32, H=32, L=4096, Lmin=100, page=16, cap=50.0, bias=1, doc=1),
        # tensor parallel by eight: few heads on the FP8 cache, distance bias, a page size that
        # is no power of two
        _attn("attn_few_heads_bias_fp8", T=24, H=8, L=6000, Lmin=1, page=48, bias=1),
        # attention weight of a small batch, bf16
        _mass("mass_small_batch_bf16", kind="bf16", T=4, L=2000, Lmin=1500),
        # attention weight of an ordinary ragged FP8 batch
        _mass("mass_batch_fp8", T=64, L=8192, Lmin=300),
        # attention weight of two long requests, bf16
        _mass("mass_long_bf16", kind="bf16", T=2, L=65536, Lmin=60000),
        # after a prefill: many requests shrink to a quarter
        _evict("evict_prefill_fp8", R=48, L=8192, Lmin=6000, budget=2048),
        # in steady decode: every request is one page above its budget
        _evict("evict_step_bf16", kind="bf16", R=256, L=1088, Lmin=1025, budget=1024, sink=4, recent=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "mass", "mass", "evict"])
    kind = rng.choice(["bf16", "fp8"])
    if op == "evict":
        R = _log_int(rng, 1, 256)
        L = _log_int(rng, 2, min(65536, max(2, 400000 // R)))
        budget = _log_int(rng, 1, L)
        sink = min(budget, rng.choice([0, 1, 4, 16]))
        return {"op": op, "kind": kind, "R": R, "L": L, "Lmin": max(1, L - _log_int(rng, 1, L)),
                "page": rng.choice([1, 16, 48, 64, 64, 128]), "budget": budget, "sink": sink,
                "recent": rng.randint(0, budget - sink)}
    T = _log_int(rng, 1, 256)
    # at most half the largest listed case's positions, so that a bf16 cache costs no more either
    L = _log_int(rng, 1, min(131072, 2000000 // T))
    return {"op": op, "kind": kind, "T": T, "H": rng.choice([1, 5, 8, 16, 32, 48, 64, 64]), "L": L,
            "Lmin": rng.choice([L, max(1, L // 2), 1]), "page": rng.choice([1, 16, 33, 48, 64, 64, 64, 128]),
            "cap": rng.choice([0.0, 0.0, 0.0, 30.0, 50.0]), "bias": rng.choice([0, 0, 1]), "doc": rng.choice([0, 0, 1])}


def _lengths(case, count):
    """Host lengths, a fixed spread over [Lmin, L]: the first request has the longest."""
    lo, hi = case["Lmin"], case["L"]
    return [hi - ((hi - lo) * ((i * 40503) % 65536)) // 65536 for i in range(count)]


def _doc_starts(case, lens):
    """First position of each token's document: none, or somewhere in the first half."""
    if not case.get("doc"):
        return [0] * len(lens)
    return [(n * ((i * 30011 + 7) % 1000)) // 2000 for i, n in enumerate(lens)]


def _cache(gen, kind, slots):
    """Latent rows of unit scale whose magnitude varies from row to row."""
    rb = ROW_FP8 if kind == "fp8" else D
    cache = torch.empty((slots, rb), dtype=torch.uint8 if kind == "fp8" else torch.bfloat16, device=DEV)
    step = 1 << 18
    for s in range(0, slots, step):
        n = min(step, slots - s)
        x = torch.randn((n, D), generator=gen, device=DEV)
        x *= torch.exp(0.25 * torch.randn((n, 1), generator=gen, device=DEV))
        x = x.to(torch.bfloat16)
        if kind == "bf16":
            cache[s:s + n] = x
            continue
        x = x.float().view(n, 2, 128)
        scale = x.abs().amax(dim=2) / 448.0
        codes = (x / scale[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, D)
        cache[s:s + n, :D] = codes
        cache[s:s + n, D:] = scale.contiguous().view(torch.uint8)
    return cache


def _pool(gen, case, lens):
    """A cache whose pages lie in random order, and the block table that names them."""
    page = case["page"]
    counts = [(n + page - 1) // page for n in lens]
    pages = sum(counts) + 8
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    width = max(counts) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = perm[at:at + c]
        at += c
    return _cache(gen, case["kind"], pages * page), table


def _slots(table, r, j, page):
    return table[r].long()[j // page] * page + j % page


def _rows(state, slot, dtype):
    """Latent rows [n, 256] of the given slots, widened exactly."""
    rows = state["cache"][slot]
    if state["case"]["kind"] == "bf16":
        return rows.to(dtype)
    codes = rows[:, :D].contiguous().view(torch.float8_e4m3fn).to(dtype).view(-1, 2, 128)
    scale = rows[:, D:].contiguous().view(torch.float32).to(dtype)
    return (codes * scale[:, :, None]).view(-1, D)


def _scores(state, t, dtype):
    """[H, n] scores of token t over its range, and the rows they come from."""
    case = state["case"]
    a, b = state["start_list"][t], state["len_list"][t]
    j = torch.arange(a, b, device=DEV)
    rows = _rows(state, _slots(state["table"], t, j, case["page"]), dtype)
    u = (state["q"][t].to(dtype) @ rows.T) * state["sm_scale"]
    if case["cap"] > 0:
        u = case["cap"] * torch.tanh(u / case["cap"])
    if case["bias"]:
        u = u - state["slopes"].to(dtype)[:, None] * (b - 1 - j).to(dtype)[None, :]
    return u, rows


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "evict":
        lens = _lengths(case, case["R"])
        cache, table = _pool(gen, case, lens)
        R, S = case["R"], case["L"] + 64
        mass = torch.exp(1.5 * torch.randn((R, S), generator=gen, device=DEV))
        # a position that no head looks at twice: some masses are equal
        mass[torch.rand((R, S), generator=gen, device=DEV) < 0.02] = 0.0625
        # token positions after earlier evictions: gaps, and the older half out of order
        pos = torch.cumsum(torch.randint(1, 4, (R, S), generator=gen, device=DEV), dim=1).to(torch.int32) - 1
        half = S // 2
        order = torch.argsort(torch.rand((R, half), generator=gen, device=DEV), dim=1)
        pos[:, :half] = torch.gather(pos[:, :half], 1, order)
        return {"case": case, "cache": cache, "table": table, "len_list": lens,
                "lengths": torch.tensor(lens, dtype=torch.int32, device=DEV), "mass": mass, "positions": pos,
                "mass_out": torch.zeros_like(mass), "positions_out": torch.zeros_like(pos)}
    T, H = case["T"], case["H"]
    lens = _lengths(case, T)
    starts = _doc_starts(case, lens)
    cache, table = _pool(gen, case, lens)
    state = {"case": case, "cache": cache, "table": table, "len_list": lens, "start_list": starts,
             "q": torch.randn((T, H, D), generator=gen, device=DEV).to(torch.bfloat16),
             "lengths": torch.tensor(lens, dtype=torch.int32, device=DEV),
             "starts": torch.tensor(starts, dtype=torch.int32, device=DEV) if case["doc"] else None,
             "slopes": (torch.exp2(-8.0 * (torch.arange(H, device=DEV) + 1) / H).float() if case["bias"] else None),
             "sm_scale": 1.0 / 16.0}
    if case["op"] == "mass":
        S = case["L"] + 64
        state["lse"] = torch.stack([torch.logsumexp(_scores(state, t, torch.float32)[0], dim=1) for t in range(T)])
        state["mass"] = torch.rand((T, S), generator=gen, device=DEV)
        state["mass_out"] = torch.zeros((T, S), device=DEV)
    return state


def _run_own(state):
    import dsa_sparse_attention_mla_gb300 as dsa

    case = state["case"]
    kind = dsa.CACHE_FP8_SCALED if case["kind"] == "fp8" else dsa.CACHE_BF16
    if case["op"] == "evict":
        lengths = torch.empty_like(state["lengths"])
        dsa.dsa_cache_evict(state["cache"], kind, state["table"], state["lengths"], state["mass"], case["budget"],
                            page_size=case["page"], sink=case["sink"], recent=case["recent"],
                            positions=state["positions"], mass_out=state["mass_out"],
                            positions_out=state["positions_out"], lengths_out=lengths)
        return {"lengths": lengths, "mass": state["mass_out"], "positions": state["positions_out"],
                "cache": state["cache"]}
    opts = {"page_size": case["page"], "starts": state["starts"], "logit_cap": case["cap"], "slopes": state["slopes"]}
    if case["op"] == "attn":
        lse = torch.empty((case["T"], case["H"]), dtype=torch.float32, device=DEV)
        out = dsa.dsa_paged_attn(state["q"], state["cache"], kind, state["table"], state["lengths"],
                                 state["sm_scale"], lse=lse, **opts)
        return {"out": out, "lse": lse}
    dsa.dsa_paged_attn_mass(state["q"], state["cache"], kind, state["table"], state["lengths"], state["sm_scale"],
                            state["lse"], state["mass"], mass_out=state["mass_out"], **opts)
    return {"mass": state["mass_out"]}


def _run_evict(state):
    case = state["case"]
    budget, sink, recent, page = case["budget"], case["sink"], case["recent"], case["page"]
    new_lens = []
    for r, n in enumerate(state["len_list"]):
        mass, pos = state["mass"][r, :n], state["positions"][r, :n]
        m = min(n, budget)
        new_lens.append(m)
        if n <= budget:
            state["mass_out"][r, :n] = mass
            state["positions_out"][r, :n] = pos
            continue
        protected = (pos < sink) | (pos > pos.max() - recent)
        key = torch.where(protected, torch.full_like(mass, math.inf), mass)
        kept = torch.zeros(n, dtype=torch.bool, device=DEV)
        kept[torch.sort(key, descending=True, stable=True).indices[:m]] = True
        movers = m + torch.argsort((~kept[m:]).to(torch.int8), stable=True)  # the kept ones first, in order
        rank = torch.cumsum(~kept[:m], dim=0) - 1
        j = torch.arange(m, device=DEV)
        src = torch.where(kept[:m], j, movers[rank.clamp(0, n - m - 1)])
        state["cache"][_slots(state["table"], r, j, page)] = state["cache"][_slots(state["table"], r, src, page)]
        state["mass_out"][r, :m] = mass[src]
        state["mass_out"][r, m:n] = 0.0
        state["positions_out"][r, :m] = pos[src]
    return {"lengths": torch.tensor(new_lens, dtype=torch.int32, device=DEV), "mass": state["mass_out"],
            "positions": state["positions_out"], "cache": state["cache"]}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "evict":
        return _run_evict(state)
    if case["op"] == "attn":
        out = torch.empty((case["T"], case["H"], D), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((case["T"], case["H"]), dtype=torch.float32, device=DEV)
        for t in range(case["T"]):
            u, rows = _scores(state, t, torch.float32)
            top = u.amax(dim=1, keepdim=True)
            e = torch.exp(u - top)
            total = e.sum(dim=1, keepdim=True)
            out[t] = ((e @ rows) / total).to(torch.bfloat16)
            lse[t] = (top + torch.log(total))[:, 0]
        return {"out": out, "lse": lse}
    for t in range(case["T"]):
        a, b = state["start_list"][t], state["len_list"][t]
        u, _ = _scores(state, t, torch.float32)
        state["mass_out"][t, a:b] = state["mass"][t, a:b] + torch.exp(u - state["lse"][t][:, None]).sum(dim=0)
    return {"mass": state["mass_out"]}


def work(case):
    row = ROW_FP8 if case["kind"] == "fp8" else 2 * D
    if case["op"] == "evict":
        nbytes = 0.0
        for n in _lengths(case, case["R"]):
            m = min(n, case["budget"])
            # mass and positions in, mass and positions out; of the m kept, the share beyond m moves
            nbytes += 8 * n + 4 * n + 4 * m + 2 * row * m * (n - m) / n + 8
        return {"bytes": int(nbytes), "flops": 0}
    lens = _lengths(case, case["T"])
    n = sum(b - a for a, b in zip(_doc_starts(case, lens), lens))
    T, H = case["T"], case["H"]
    if case["op"] == "attn":
        return {"bytes": n * row + T * H * D * 4 + T * H * 4, "flops": 2 * n * H * 2 * D}
    return {"bytes": n * (row + 8) + T * H * D * 2 + T * H * 4, "flops": 2 * n * H * D}


def exact(case, seed):
    """The definitions in 64 bits."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "evict":
        import numpy as np

        mass, pos = st["mass"].cpu().numpy(), st["positions"].cpu().numpy()
        mass_out, pos_out = np.zeros_like(mass), np.zeros_like(pos)
        lens = []
        table = st["table"].cpu().numpy()
        src_slots, dst_slots = [], []
        for r, n in enumerate(st["len_list"]):
            b = case["budget"]
            if n <= b:
                mass_out[r, :n], pos_out[r, :n] = mass[r, :n], pos[r, :n]
                lens.append(n)
                continue
            newest = pos[r, :n].max()
            rank = mass[r, :n].astype(np.float64)
            rank[(pos[r, :n] < case["sink"]) | (pos[r, :n] > newest - case["recent"])] = np.inf
            best = np.lexsort((np.arange(n), -rank))[:b]
            alive = np.zeros(n, dtype=bool)
            alive[best] = True
            at = np.arange(n)
            at[:b][~alive[:b]] = np.flatnonzero(alive[b:]) + b
            mass_out[r, :b], pos_out[r, :b] = mass[r, at[:b]], pos[r, at[:b]]
            lens.append(b)
            moved = np.flatnonzero(at[:b] != np.arange(b))
            p = case["page"]
            dst_slots.append(table[r, moved // p].astype(np.int64) * p + moved % p)
            src_slots.append(table[r, at[moved] // p].astype(np.int64) * p + at[moved] % p)
        if src_slots:
            src = torch.from_numpy(np.concatenate(src_slots)).to(DEV)
            dst = torch.from_numpy(np.concatenate(dst_slots)).to(DEV)
            st["cache"][dst] = st["cache"][src]
        return {"lengths": torch.tensor(lens, dtype=torch.int32), "mass": torch.from_numpy(mass_out),
                "positions": torch.from_numpy(pos_out), "cache": st["cache"]}
    page, cap = case["page"], case["cap"]
    outs, lses = [], []
    mass = st["mass_out"].to(f64) if case["op"] == "mass" else None
    for t, (a, b) in enumerate(zip(st["start_list"], st["len_list"])):
        at = torch.arange(a, b, device=DEV)
        slot = st["table"][t, torch.div(at, page, rounding_mode="floor")].to(torch.int64) * page + at.remainder(page)
        raw = st["cache"].index_select(0, slot)
        if case["kind"] == "fp8":
            code = raw[:, :D].contiguous().view(torch.float8_e4m3fn).to(torch.float32).to(f64)
            k = code * raw[:, D:].contiguous().view(torch.float32).to(f64).repeat_interleave(128, dim=1)
        else:
            k = raw.to(f64)
        s = torch.einsum("hd,nd->hn", st["q"][t].to(f64), k) * st["sm_scale"]
        if cap > 0:
            s = torch.tanh(s / cap) * cap
        if case["bias"]:
            s -= st["slopes"].to(f64).view(-1, 1) * (b - 1 - at).view(1, -1)
        if mass is not None:
            mass[t, a:b] = st["mass"][t, a:b].to(f64) + torch.exp(s - st["lse"][t].to(f64).view(-1, 1)).sum(0)
            continue
        lse = torch.logsumexp(s, dim=1)
        lses.append(lse)
        outs.append(torch.einsum("hn,nd->hd", torch.exp(s - lse[:, None]), k))
    if mass is not None:
        return {"mass": mass}
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
