"""Eviction from the paged cache on the GPU, against the definition (oracle/paged.py): lengths,
masses, positions and every cache byte equal; and the loop attention -> mass -> eviction."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from oracle import paged as R

pytestmark = pytest.mark.gpu

BF16, FP8 = dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED
GEOMETRY = {(BF16, 256): 512, (FP8, 256): 264, (BF16, 512): 1152, (FP8, 512): 656}


def build(rng, lens, S, page, row):
    """(cache bytes, block table, mass, positions): scattered pages, masses with ties, zeros and infinities."""
    need = [(max(n, 0) + page - 1) // page for n in lens]
    pages = sum(need) + 2
    perm = rng.permutation(pages)
    bt = np.full((len(lens), max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for r, c in enumerate(need):
        bt[r, :c] = perm[at:at + c]
        at += c
    cache = rng.integers(0, 256, size=(pages * page, row), dtype=np.uint8)
    mass = rng.random((len(lens), S)).astype(np.float32)
    mass[rng.random(mass.shape) < 0.3] = 0.5
    mass[rng.random(mass.shape) < 0.1] = 0.0
    mass[rng.random(mass.shape) < 0.05] = -0.0
    mass[rng.random(mass.shape) < 0.02] = np.inf
    mass[rng.random(mass.shape) < 0.02] *= -1
    pos = np.stack([rng.permutation(3 * S)[:S] for _ in lens]).astype(np.int32)
    return cache, bt, mass, pos


def as_cache(raw, kind, dev):
    t = torch.from_numpy(raw).to(dev)
    return t if kind == FP8 else t.view(torch.bfloat16)


def check(dev, lens, budgets, S, page=64, kind=FP8, d=256, sink=0, recent=0, seed=0, inplace=False, use_pos=True,
          scalar=False):
    rng = np.random.default_rng(seed)
    raw, bt, mass, pos = build(rng, lens, S, page, GEOMETRY[kind, d])
    ref = R.evict(lens, budgets, mass, pos if use_pos else None, sink, recent)
    want = raw.copy()
    for r, (_, moves, _, _) in enumerate(ref):
        for s, t in moves:
            want[bt[r, t // page] * page + t % page] = raw[bt[r, s // page] * page + s % page]
    cache = as_cache(raw, kind, dev)
    m, p = torch.from_numpy(mass).to(dev), torch.from_numpy(pos).to(dev) if use_pos else None
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kw = {"budget": budgets[0]} if scalar else {"budgets": torch.tensor(budgets, dtype=torch.int32, device=dev)}
    if not inplace:
        kw.update(mass_out=torch.full_like(m, -3.0), lengths_out=torch.full_like(ln, -3),
                  positions_out=torch.full((len(lens), S), -3, dtype=torch.int32, device=dev))
    l2, m2, p2 = dsa.dsa_cache_evict(cache, kind, torch.from_numpy(bt).to(dev), ln, m, page_size=page, sink=sink,
                                     recent=recent, positions=p, d_nope=d, d_rope=64 if d == 512 else 0, error_word=err,
                                     **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert l2.cpu().tolist() == [x[0] for x in ref]
    got_m, got_p = m2.cpu().numpy(), None if p2 is None else p2.cpu().numpy()
    for r, (_, _, mr, pr) in enumerate(ref):
        n = max(lens[r], 0)
        b = min(n, max(budgets[r], 0))
        assert np.array_equal(got_m[r, :n].view(np.uint32), mr[:n].view(np.uint32)), r
        if got_p is not None:
            assert np.array_equal(got_p[r, :b], pr[:b]), r
        if inplace:
            assert np.array_equal(got_m[r, n:].view(np.uint32), mass[r, n:].view(np.uint32))
        else:
            assert (got_m[r, n:] == -3.0).all() and (got_p is None or (got_p[r, n:] == -3).all())
    assert np.array_equal(cache.cpu().view(torch.uint8).numpy(), want)


LENS = [0, 1, 2, 63, 64, 65, 513, 1000, 1025]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("use_pos", [False, True])
@pytest.mark.parametrize("budget", [0, 1, 64, 511, 512, 1024])
def test_ragged(gpu, budget, use_pos, inplace):
    check(gpu, LENS, [budget] * len(LENS), 1100, sink=min(4, budget), recent=budget // 4, seed=budget, inplace=inplace,
          use_pos=use_pos, scalar=True)


@pytest.mark.parametrize("kind,d", list(GEOMETRY))
@pytest.mark.parametrize("page", [1, 7, 16, 64, 256])
def test_geometries_and_pages(gpu, kind, d, page):
    check(gpu, [300, 777, 5], [100, 700, 2], 800, page=page, kind=kind, d=d, sink=3, recent=20, seed=page)


@pytest.mark.parametrize("lens,budgets", [([20000], [4097]), ([20000], [19999]), ([70001], [35000]),
                                          ([4096] * 3, [4095, 1, 4096]), ([9000, 100, 9000], [-5, 200, 4500])])
def test_long(gpu, lens, budgets):
    check(gpu, lens, budgets, max(lens) + 3, kind=BF16, sink=4, recent=50, seed=sum(lens))


def test_all_equal_and_all_protected(gpu):
    """Ties alone decide: the lowest positions stay; protected positions past the budget rank equal."""
    rng = np.random.default_rng(0)
    raw, bt, mass, pos = build(rng, [900], 900, 64, 264)
    for m in (np.full_like(mass, 0.25), np.zeros_like(mass)):
        lens, out, p = dsa.dsa_cache_evict(
            torch.from_numpy(raw).to(gpu), FP8, torch.from_numpy(bt).to(gpu),
            torch.tensor([900], dtype=torch.int32, device=gpu), torch.from_numpy(m).to(gpu), 300, page_size=64,
            positions_out=torch.zeros((1, 900), dtype=torch.int32, device=gpu))
        assert p[0, :300].cpu().tolist() == list(range(300))
    check(gpu, [900], [100], 900, sink=900, recent=900, seed=9)
    check(gpu, [900], [100], 900, sink=0, recent=2 ** 31 - 1, seed=9)


@pytest.mark.parametrize("what", ["length past the rows", "length past the table", "negative page", "page past the pool"])
def test_bad_requests_keep_everything(gpu, what):
    rng = np.random.default_rng(4)
    raw, bt, mass, pos = build(rng, [500, 500], 512, 64, 264)
    lens = [500, 500]
    if what == "length past the rows":
        lens[0] = 513
    elif what == "length past the table":
        bt = bt[:, :7].copy()
    elif what == "negative page":
        bt[0, 3] = -1
    else:
        bt[0, 3] = len(raw) // 64
    one = what != "length past the table"
    cache = torch.from_numpy(raw).to(gpu)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    ln = torch.tensor(lens, dtype=torch.int32, device=gpu)
    l2, m2, p2 = dsa.dsa_cache_evict(cache, FP8, torch.from_numpy(bt).to(gpu), ln, torch.from_numpy(mass).to(gpu), 128,
                                     page_size=64, positions=torch.from_numpy(pos).to(gpu),
                                     mass_out=torch.zeros((2, 512), device=gpu),
                                     positions_out=torch.zeros((2, 512), dtype=torch.int32, device=gpu),
                                     lengths_out=torch.zeros(2, dtype=torch.int32, device=gpu), error_word=err)
    torch.cuda.synchronize()
    assert err.item() == dsa.DEVERR_INDEX_OUT_OF_RANGE
    assert l2.cpu().tolist() == [lens[0], 128 if one else 500]
    n = min(lens[0], 512)
    assert np.array_equal(m2.cpu().numpy()[0, :n], mass[0, :n]) and np.array_equal(p2.cpu().numpy()[0, :n], pos[0, :n])
    got = cache.cpu().numpy()
    moved = np.flatnonzero((got != raw).any(axis=1))
    mine = set((np.asarray(build(np.random.default_rng(4), [500, 500], 512, 64, 264)[1])[1][:, None] * 64 +
                np.arange(64)).ravel()) if one else set()
    assert set(moved) <= mine


def test_strided_rows(gpu):
    rng = np.random.default_rng(6)
    raw, bt, mass, pos = build(rng, [300, 200], 320, 64, 264)
    ref = R.evict([300, 200], [64, 64], mass, pos, 2, 8)
    big_m = torch.full((2, 400), 9.0, device=gpu)
    big_p = torch.full((2, 350), 9, dtype=torch.int32, device=gpu)
    big_m[:, :320], big_p[:, :320] = torch.from_numpy(mass).to(gpu), torch.from_numpy(pos).to(gpu)
    dsa.dsa_cache_evict(torch.from_numpy(raw).to(gpu), FP8, torch.from_numpy(bt).to(gpu),
                        torch.tensor([300, 200], dtype=torch.int32, device=gpu), big_m[:, :320], 64, page_size=64, sink=2,
                        recent=8, positions=big_p[:, :320])
    torch.cuda.synchronize()
    for r, n in enumerate([300, 200]):
        assert np.array_equal(big_m[r, :n].cpu().numpy(), ref[r][2][:n])
        assert np.array_equal(big_p[r, :64].cpu().numpy(), ref[r][3][:64])
    assert (big_m[:, 320:] == 9).all() and (big_p[:, 320:] == 9).all()


def test_graph_replay(gpu):
    rng = np.random.default_rng(8)
    raw, bt, mass, pos = build(rng, [700, 650], 700, 64, 264)
    cache0 = torch.from_numpy(raw).to(gpu)
    m0, p0 = torch.from_numpy(mass).to(gpu), torch.from_numpy(pos).to(gpu)
    l0 = torch.tensor([700, 650], dtype=torch.int32, device=gpu)
    t = torch.from_numpy(bt).to(gpu)

    def call(c, m, p, ln):
        return dsa.dsa_cache_evict(c, FP8, t, ln, m, 256, page_size=64, sink=4, recent=32, positions=p)

    c1, m1, p1, l1 = cache0.clone(), m0.clone(), p0.clone(), l0.clone()
    call(c1, m1, p1, l1)
    c2, m2, p2, l2 = cache0.clone(), m0.clone(), p0.clone(), l0.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c2, m2, p2, l2)
    for _ in range(3):
        c2.copy_(cache0), m2.copy_(m0), p2.copy_(p0), l2.copy_(l0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c1, c2) and torch.equal(m1.view(torch.int32), m2.view(torch.int32))
        assert torch.equal(p1, p2) and torch.equal(l1, l2)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_decode_loop_with_eviction(gpu, kind):
    """Steps as a server runs them: pack a new row, attend, add the weights to the mass, evict down
    to the budget when a page fills. The attention after each eviction equals the fp64 attention
    over the rows a host-side copy of the bookkeeping keeps."""
    import oracle as O
    from oracle import projection as P

    rng = np.random.default_rng(77)
    Rq, S, budget, page, H = 3, 256, 128, 64, 16
    bt = torch.from_numpy(rng.permutation(Rq * 4).reshape(Rq, 4).astype(np.int32)).to(gpu)
    slots = Rq * 4 * page
    cache = (torch.zeros((slots, 264), dtype=torch.uint8, device=gpu) if kind == FP8
             else torch.zeros((slots, 256), dtype=torch.bfloat16, device=gpu))
    mass = torch.zeros((Rq, S), device=gpu)
    positions = torch.zeros((Rq, S), dtype=torch.int32, device=gpu)
    lengths = torch.zeros(Rq, dtype=torch.int32, device=gpu)
    host = [[] for _ in range(Rq)]   # (token position, row) in cache order
    host_len = [0] * Rq
    table = bt.cpu().numpy()
    evictions = 0
    for step in range(330):
        rows = P.f64_to_bf16(rng.standard_normal((Rq, 256)))
        loc = np.array([table[r, host_len[r] // page] * page + host_len[r] % page for r in range(Rq)], dtype=np.int64)
        dev_rows = torch.from_numpy(rows.view(np.int16)).view(torch.bfloat16).to(gpu)
        dev_loc = torch.from_numpy(loc).to(gpu)
        if kind == FP8:
            dsa.dsa_quant_k_cache(dev_rows, out_loc=dev_loc, cache=cache)
        else:
            cache[dev_loc] = dev_rows
        positions[torch.arange(Rq, device=gpu), lengths.long()] = step
        lengths += 1
        for r in range(Rq):
            host[r].append((step, rows[r]))
            host_len[r] += 1
        q = P.f64_to_bf16(rng.standard_normal((Rq, H, 256)))
        dq = torch.from_numpy(q.view(np.int16)).view(torch.bfloat16).to(gpu)
        lse = torch.empty((Rq, H), device=gpu)
        out = dsa.dsa_paged_attn(dq, cache, kind, bt, lengths, 1 / 16, page_size=page, lse=lse)
        dsa.dsa_paged_attn_mass(dq, cache, kind, bt, lengths, 1 / 16, lse, mass, page_size=page)
        if step % 47 == 0 or step > 320:
            torch.cuda.synchronize()
            for r in range(Rq):
                b = np.stack([x[1] for x in host[r]])
                c = b if kind == BF16 else O.quant_k_cache(b, num_slots=len(b))
                u, k, _, _ = R.scores(P.bf16_to_f64(q[r]), c, None, 1, 0, 0, len(b), 1 / 16)
                ref, rl, _, l2 = R.softmax_output(u, k)
                e = np.abs(out[r].float().cpu().numpy() - ref)
                assert np.linalg.norm(e) <= 2.0 ** -7 * (np.linalg.norm(ref) + np.linalg.norm(l2))
            assert np.array_equal(np.sort(positions.cpu().numpy()[:, :host_len[0]], axis=1),
                                  np.array([sorted(x[0] for x in host[r]) for r in range(Rq)]))
        if host_len[0] == budget + page:
            m = mass.cpu().numpy()
            p = positions.cpu().numpy()
            plan = R.evict(host_len, [budget] * Rq, m, p, 4, 32)
            dsa.dsa_cache_evict(cache, kind, bt, lengths, mass, budget, page_size=page, sink=4, recent=32,
                                positions=positions)
            for r in range(Rq):
                for s, d in plan[r][1]:
                    host[r][d] = host[r][s]
                host[r] = host[r][:budget]
                host_len[r] = budget
            torch.cuda.synchronize()
            assert lengths.cpu().tolist() == host_len
            evictions += 1
    assert evictions >= 3


def test_two_evictions_at_once(gpu):
    """On two streams, then from two captured graphs on two streams: each keeps its own lists."""
    rng = np.random.default_rng(12)
    states = []
    for lens, S, b in (([5000, 4100, 9], 5000, 1500), ([900] * 40, 1000, 333)):  # both select variants
        raw, bt, mass, pos = build(rng, lens, S, 64, 264)
        start = [torch.from_numpy(raw).to(gpu), torch.from_numpy(mass).to(gpu), torch.from_numpy(pos).to(gpu),
                 torch.tensor(lens, dtype=torch.int32, device=gpu)]
        states.append({"table": torch.from_numpy(bt).to(gpu), "start": start, "b": b, "now": [x.clone() for x in start]})

    def call(s):
        c, m, p, ln = s["now"]
        dsa.dsa_cache_evict(c, FP8, s["table"], ln, m, s["b"], page_size=64, sink=2, recent=16, positions=p)

    def reset():
        for s in states:
            for x, x0 in zip(s["now"], s["start"]):
                x.copy_(x0)
        torch.cuda.synchronize()

    for s in states:
        call(s)
    torch.cuda.synchronize()
    want = [[x.clone() for x in s["now"]] for s in states]
    assert [w[3].max().item() for w in want] == [1500, 333]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, s in zip(graphs, states):
        reset()
        with torch.cuda.graph(g):
            call(s)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for go in (lambda i: call(states[i]), lambda i: graphs[i].replay()):
        for _ in range(4):
            reset()
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    go(i)
            torch.cuda.synchronize()
            for s, w in zip(states, want):
                for x, y in zip(s["now"], w):
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
