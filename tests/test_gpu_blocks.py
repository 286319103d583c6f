"""Block means, block scores and the choice of blocks on the GPU against oracle/steps.py, and the step
plan -> norms -> means -> scores -> choice -> attention as a whole.

Tolerances. Means: fp32 sums of n rows err by at most n * 2^-24 of the mean |row|, rounding to bf16 by
half a step, 2^-8 |mean|. Scores: bf16 products are exact; an fp32 accumulator that truncates errs by
less than 2^-23 of the sum of |q s| at each of at most 256 additions, which a weighted sum over the
heads carries along; that sum errs by (H + 2) * 2^-24 of its terms."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from oracle import paged as G
from oracle import steps as S

pytestmark = pytest.mark.gpu

BF16, FP8 = dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED
BAD = dsa.DEVERR_INDEX_OUT_OF_RANGE


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


def raw(cache):
    c = cache.cpu()
    return c.numpy() if c.dtype == torch.uint8 else c.view(torch.int16).numpy().view(np.uint16)


def tables(rng, lens, page, spare=3, cols=2):
    """(table, pages of the pool): scattered pages for these lengths."""
    need = [-(-max(int(n), 0) // page) for n in lens]
    perm = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need + [0]) + cols), -1, dtype=np.int32)
    at = 0
    for r, c in enumerate(need):
        table[r, :c] = perm[at:at + c]
        at += c
    return table, sum(need) + spare


def make_cache(dev, kind, slots, seed):
    gen = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((slots, 256), generator=gen, device=dev) * torch.exp(torch.randn((slots, 1), generator=gen, device=dev))
    x = x.to(torch.bfloat16)
    return x if kind == BF16 else dsa.dsa_quant_k_cache(x)


# --------------------------------------------------------------------------------------- means --
def check_pool(dev, lens, new, page, kind, seed=0, pad=0, poison=False):
    rng = np.random.default_rng(seed)
    table, pages = tables(rng, lens, page)
    cache = make_cache(dev, kind, pages * page, seed)
    if poison:  # NaN in every row at or past its request's length
        for r, n in enumerate(lens):
            for j in range(n, -(-n // page) * page):
                slot = table[r, j // page] * page + j % page
                cache[slot] = 0x7F if kind == FP8 else float("nan")
                if kind == FP8:
                    cache[slot, 256:] = 0xFF
    req = [r for r, m in enumerate(new) for _ in range(m)] + [0] * pad
    pos = [n - m + i for n, m in zip(lens, new) for i in range(m)] + [-1] * pad
    summary = torch.full((pages, 256), 3.0, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    args = (cache, kind, i32(table, dev), i32(pos, dev), i32(lens, dev), summary)
    dsa.dsa_block_pool(*args, page_size=page, req_of_token=i32(req, dev), error_word=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    want = S.pool(raw(cache), table, page, req, pos, lens)
    got = f64(summary)
    for p in range(pages):
        if p not in want:
            assert (got[p] == 3.0).all()
            continue
        mean, size, n = want[p]
        tol = size * n * 2.0 ** -24 + np.abs(mean) * 2.0 ** -8 * (1 + 2.0 ** -10) + 1e-37
        assert (np.abs(got[p] - mean) <= tol).all(), p
    again = torch.full_like(summary, 3.0)
    dsa.dsa_block_pool(*args[:-1], again, page_size=page, req_of_token=i32(req, dev))
    assert torch.equal(again, summary)


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("page", [1, 16, 33, 64, 200])
def test_pool(gpu, page, kind):
    check_pool(gpu, [1], [1], page, kind)
    check_pool(gpu, [1, 64, 65, 500, 17], [1, 1, 1, 1, 1], page, kind, poison=page > 1)
    check_pool(gpu, [300, 5, 129], [300, 0, 70], page, kind, pad=9, poison=page > 1)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_pool_of_many_tokens(gpu, kind):
    check_pool(gpu, [3000, 40, 2000], [3000, 40, 1500], 64, kind, pad=70)  # more than 4096 with the padding
    check_pool(gpu, [7] * 4200, [1] * 4200, 8, kind)  # a decode step of so many requests


def test_pool_without_a_request_map(gpu):
    cache = make_cache(gpu, BF16, 64, 1)
    summary = torch.zeros((4, 256), dtype=torch.bfloat16, device=gpu)
    dsa.dsa_block_pool(cache, BF16, i32([[2], [0]], gpu), i32([0, 15], gpu), i32([1, 16], gpu), summary, page_size=16)
    assert torch.equal(summary[2], cache[32])
    assert (summary[0].float() - cache[:16].float().mean(0)).abs().max() < 0.05 and (summary[[1, 3]] == 0).all()


def test_pool_bad_entries_are_skipped(gpu):
    cache = make_cache(gpu, FP8, 64, 1)
    table = i32([[2, 4, -1, 3], [0, 1, 1, 0]], gpu)

    def run(pos, req, lens=(64, 20)):
        summary = torch.zeros((4, 256), dtype=torch.bfloat16, device=gpu)
        err = torch.zeros(1, dtype=torch.int32, device=gpu)
        dsa.dsa_block_pool(cache, FP8, table, i32(pos, gpu), i32(lens, gpu), summary, page_size=16, req_of_token=i32(req, gpu),
                           error_word=err)
        return summary.ne(0).any(1).nonzero().flatten().tolist(), err.item()

    assert run([3, 50], [0, 0]) == ([2, 3], 0)
    assert run([3, 17], [0, 0]) == ([2], BAD)  # page 4 of 4
    assert run([33, 3], [0, 1]) == ([0], BAD)  # page -1
    assert run([64, 3], [0, 1]) == ([0], BAD)  # past the table
    assert run([2 ** 31 - 1, 3], [0, 1]) == ([0], BAD)
    assert run([3, 3], [2, 1]) == ([0], BAD) and run([3, 3], [-1, 1]) == ([0], BAD)  # no such request
    assert run([3, 33], [0, 1]) == ([2], BAD)  # a block with no cached position
    assert run([-1, -7], [0, 5]) == ([], 0)  # padding
    # the page's rows end at the cache's last slot
    summary = torch.zeros((5, 256), dtype=torch.bfloat16, device=gpu)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    for n, bits in ((1, 0), (9, BAD)):
        dsa.dsa_block_pool(cache[:56], FP8, i32([[3]], gpu), i32([0], gpu), i32([n], gpu), summary, page_size=16, error_word=err)
        assert err.item() == bits


# -------------------------------------------------------------------------------------- scores --
def check_scores(dev, tokens, H, page=64, weights=False, seed=0, scale=1 / 16, summary_scale=1.0, strided=False, lens=None,
                 pool=None, more_cols=0, qscale=1.0):
    """tokens: (request, length) pairs."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    R = max(r for r, _ in tokens) + 1
    most = [max([n for q, n in tokens if q == r] + [0]) for r in range(R)]
    table, pages = tables(rng, most, page)
    T, width = len(tokens), table.shape[1] + more_cols
    summary = (torch.randn((pages, 256), generator=gen, device=dev) * summary_scale).to(torch.bfloat16)
    used = np.unique(table[table >= 0])
    summary[np.setdiff1d(np.arange(pages), used)] = float("nan")  # pages that no token names
    if strided:
        big = torch.full((T, H + 2, 264), float("nan"), dtype=torch.bfloat16, device=dev)
        q = big[:, 1:H + 1, :256]
    else:
        q = torch.empty((T, H, 256), dtype=torch.bfloat16, device=dev)
    q.copy_(torch.randn((T, H, 256), generator=gen, device=dev) * qscale)
    w = torch.randn((T, H), generator=gen, device=dev) if weights else None
    out = torch.full((T, width + (5 if strided else 0)), 77.0, device=dev)[:, :width]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    run = lambda o: dsa.dsa_block_scores(  # noqa: E731
        q, summary, i32(table, dev), i32([n for _, n in tokens], dev), scale, page_size=page,
        req_of_token=i32([r for r, _ in tokens], dev), weights=w, out=o, error_word=err)
    assert run(out) is out
    torch.cuda.synchronize()
    assert err.item() == 0
    got, qd, sd, wd = f64(out), f64(q), f64(summary), None if w is None else f64(w)
    scale = float(np.float32(scale))
    for t, (r, n) in enumerate(tokens):
        nb = -(-max(n, 0) // page)
        assert (got[t, nb:] == 77.0).all(), t
        want, size, terms = S.scores(qd[t], sd, table[r, :nb], scale, None if wd is None else wd[t])
        tol = size * 256 * 2.0 ** -23 + terms * (H + 2) * 2.0 ** -24 + 1e-37
        off = np.abs(got[t, :nb] - want) - tol
        assert nb == 0 or off.max() <= 0, (t, int(off.argmax()), got[t, off.argmax()], want[off.argmax()])
    again = torch.full_like(out, 77.0)
    run(again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("H", [1, 3, 8, 16, 33, 48, 64, 65, 127, 128])
def test_scores_heads(gpu, H, weights):
    check_scores(gpu, [(0, 700), (1, 64), (2, 65), (3, 0), (4, 1), (5, 9000)], H, weights=weights, seed=H)


@pytest.mark.parametrize("page", [1, 7, 16, 64, 128])
def test_scores_pages_and_lengths(gpu, page):
    check_scores(gpu, [(0, 1), (1, page), (2, page + 1), (3, 128 * page), (4, 128 * page + 1), (5, 127 * page), (6, -3)], 16,
                 page, weights=True, seed=page, more_cols=3)


@pytest.mark.parametrize("H", [8, 20, 64, 128])
def test_scores_of_a_prefill_chunk(gpu, H):
    """Neighbouring tokens of one request, in chunks whose borders fall anywhere in a tile of tokens."""
    chunk = lambda r, a, b: [(r, n) for n in range(a, b)]  # noqa: E731
    check_scores(gpu, chunk(0, 3000, 3009), H, 16, weights=True)
    check_scores(gpu, chunk(0, 1, 40) + chunk(1, 4000, 4003) + chunk(2, 250, 290) + [(0, 5)], H, 16, seed=1)
    check_scores(gpu, [(0, 0)] * 6 + chunk(1, 2040, 2051) + [(0, 0)] * 3, H, 16, seed=2)


def test_scores_requests_in_any_order(gpu):
    rng = np.random.default_rng(5)
    check_scores(gpu, [(int(r), int(n)) for r, n in zip(rng.integers(0, 4, 61), rng.integers(0, 3000, 61))], 24, 16,
                 weights=True)


def test_scores_strides_and_magnitudes(gpu):
    toks = [(0, 900), (0, 901), (1, 300), (2, 2000)]
    check_scores(gpu, toks, 12, strided=True, weights=True)
    check_scores(gpu, toks, 64, strided=True)
    check_scores(gpu, toks, 64, summary_scale=1e-15, qscale=1e-10, scale=1e-3)
    check_scores(gpu, toks, 64, summary_scale=1e12, qscale=1e12, scale=3.0, weights=True)


def test_scores_of_a_large_batch(gpu):
    rng = np.random.default_rng(6)
    check_scores(gpu, [(r, int(n)) for r, n in enumerate(rng.integers(0, 3000, 400))], 8, 16)
    check_scores(gpu, [(0, n) for n in range(5000, 7500, 3)], 16, 64, weights=True)


@pytest.mark.parametrize("H,page,top", [(64, 64, 8000), (64, 16, 5000), (64, 16, 2047), (64, 16, 9000), (128, 16, 9000),
                                        (32, 16, 6200), (48, 16, 4100), (48, 16, 12000), (8, 16, 30000)])
@pytest.mark.parametrize("weights", [False, True])
def test_scores_of_many_groups(gpu, H, page, top, weights):
    """Enough tokens that a group fills an MMA: units of one tile, of odd numbers of tiles and of tokens of several
    requests follow one another, over many rounds of every ring. Run often: the warps' order differs."""
    gen = torch.Generator(device=gpu).manual_seed(top + H)
    T, R = 6000, 3
    lens = torch.randint(0, top, (T,), generator=gen, device=gpu).to(torch.int32)
    lens[:2000] = torch.arange(2000, device=gpu).to(torch.int32) + top - 2000 if top > 4000 else lens[:2000]
    lens[3000:3500] = 0
    lens[3500:4200] = lens[3500:4200] % (128 * page)  # one tile, between groups of several
    req = torch.zeros(T, dtype=torch.int32, device=gpu)
    req[2500:] = 1
    req[5000:] = torch.randint(0, R, (1000,), generator=gen, device=gpu).to(torch.int32)
    nb = -(-top // page)
    table = torch.randperm(R * nb, generator=gen, device=gpu).to(torch.int32).view(R, nb)
    summary = torch.randn((R * nb, 256), generator=gen, device=gpu).to(torch.bfloat16)
    q = torch.randn((T, H, 256), generator=gen, device=gpu).to(torch.bfloat16)
    w = torch.randn((T, H), generator=gen, device=gpu) if weights else None
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    outs = [torch.full((T, nb), 7.0, device=gpu) for _ in range(8)]
    for out in outs:
        dsa.dsa_block_scores(q, summary, table, lens, 0.125, page_size=page, req_of_token=req, weights=w, out=out, error_word=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert all(torch.equal(o, outs[0]) for o in outs)
    step = 500
    for a in range(0, T, step):
        x = q[a:a + step].double()
        for r in req[a:a + step].unique().tolist():
            s = summary[table[r].long()].double()
            dot = torch.einsum("thd,bd->thb", x, s).clamp_(min=0) * 0.125
            ww = torch.ones((step, H), dtype=torch.float64, device=gpu) if w is None else w[a:a + step].double()
            want = torch.einsum("thb,th->tb", dot, ww)
            # |q| |s| bounds the sum of products of each head
            size = 0.125 * (ww.abs() * x.norm(dim=2)).sum(1)[:, None] * s.norm(dim=1)[None, :]
            tol = size * (256 * 2.0 ** -23 + (H + 2) * 2.0 ** -24)
            mine = req[a:a + step] == r
            live = (torch.arange(nb, device=gpu)[None] * page < lens[a:a + step, None]) & mine[:, None]
            got = outs[0][a:a + step].double()
            assert ((got - want).abs() <= tol)[live].all()
            assert (got == 7.0)[~live & mine[:, None]].all()


def test_scores_bad_entries(gpu):
    q = torch.ones((3, 4, 256), dtype=torch.bfloat16, device=gpu)
    summary = torch.ones((4, 256), dtype=torch.bfloat16, device=gpu)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)

    def run(table, lens, req=None, width=None):
        out = torch.full((3, width or len(table[0])), 5.0, device=gpu)
        err.zero_()
        dsa.dsa_block_scores(q, summary, i32(table, gpu), i32(lens, gpu), 1.0, page_size=16, out=out, error_word=err,
                             req_of_token=None if req is None else i32(req, gpu))
        return out.tolist(), err.item()

    inf, full = float("inf"), 4 * 256.0
    good = [[0, 1], [2, 3], [1, 1]]
    assert run(good, [32, 17, 1]) == ([[full, full], [full, full], [full, 5.0]], 0)
    assert run([[0, 4], [-1, 3], [2 ** 31 - 1, -2 ** 31]], [32, 32, 32]) == (
        [[full, -inf], [-inf, full], [-inf, -inf]], BAD)
    assert run(good, [33, 2 ** 31 - 1, 16]) == ([[full, full], [full, full], [full, 5.0]], BAD)
    assert run(good, [32, 32, 32], [0, 3, -1]) == ([[full, full], [5.0, 5.0], [5.0, 5.0]], BAD)
    assert run(good, [32, 16, 32], width=1) == ([[full], [full], [full]], BAD)


def test_scores_infinities_and_nan(gpu):
    """NaN and infinities of a page reach its own block's score only; NaN passes through the maximum."""
    q = torch.ones((2, 4, 256), dtype=torch.bfloat16, device=gpu)
    q[1, 2, 7] = float("nan")
    summary = torch.ones((6, 256), dtype=torch.bfloat16, device=gpu)
    summary[1, 3], summary[2, 9], summary[3] = float("nan"), float("inf"), -1.0
    summary[4, 100] = -float("inf")
    got = dsa.dsa_block_scores(q, summary, i32([[0, 1, 2, 3, 4, 5]], gpu), i32([96, 96], gpu), 1.0, page_size=16,
                               req_of_token=i32([0, 0], gpu)).cpu()
    inf = float("inf")
    assert got[0, [0, 2, 3, 4, 5]].tolist() == [1024.0, inf, 0.0, 0.0, 1024.0] and got[0, 1].isnan()
    assert got[1].isnan().all()


def test_scores_streams_and_graphs(gpu):
    gen = torch.Generator(device=gpu).manual_seed(9)
    q = torch.randn((40, 64, 256), generator=gen, device=gpu).to(torch.bfloat16)
    summary = torch.randn((300, 256), generator=gen, device=gpu).to(torch.bfloat16)
    table, lens = i32(np.arange(300).reshape(1, 300), gpu), torch.arange(40, dtype=torch.int32, device=gpu) * 120 + 1
    req = torch.zeros(40, dtype=torch.int32, device=gpu)
    run = lambda: dsa.dsa_block_scores(q, summary, table, lens, 0.1, page_size=16, req_of_token=req)  # noqa: E731
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    third = run()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    lens.copy_(lens.flip(0))
    want = run()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_pages_past_four_gigabytes(gpu):
    """Cache rows and summaries whose offsets pass 32 bits."""
    page = 64
    pages = (1 << 32) // 512 + 200
    rows = (1 << 32) // 264 + 64 * page
    far = rows // page - 1
    cache = torch.zeros((rows, 264), dtype=torch.uint8, device=gpu)
    part = make_cache(gpu, FP8, 4 * page, 3)
    picks = [far, 0, far - 1, 7]
    for i, p in enumerate(picks):
        cache[p * page:(p + 1) * page] = part[i * page:(i + 1) * page]
    summary = torch.zeros((pages, 256), dtype=torch.bfloat16, device=gpu)
    lens = i32([4 * page], gpu)
    table = i32([picks], gpu)
    pos, req = i32([0, 64, 128, 192], gpu), i32([0, 0, 0, 0], gpu)
    dsa.dsa_block_pool(cache, FP8, table, pos, lens, summary, page_size=page, req_of_token=req)
    small = torch.zeros((4, 256), dtype=torch.bfloat16, device=gpu)
    dsa.dsa_block_pool(part, FP8, i32([[0, 1, 2, 3]], gpu), pos, lens, small, page_size=page, req_of_token=req)
    assert torch.equal(summary[picks], small) and small.ne(0).any(1).all()
    ends = [pages - 1, 5, pages - 60, pages - 2]
    summary[ends] = small
    q = torch.randn((2, 16, 256), device=gpu).to(torch.bfloat16)
    args = dict(lengths=i32([4 * page, 3 * page], gpu), sm_scale=0.5, page_size=page, req_of_token=i32([0, 0], gpu))
    got = dsa.dsa_block_scores(q, summary, i32([ends], gpu), **args)
    assert torch.equal(got, dsa.dsa_block_scores(q, small, i32([[0, 1, 2, 3]], gpu), **args))


# -------------------------------------------------------------------------------------- choice --
def rows_of(rng, T, width):
    s = np.exp(rng.standard_normal((T, width))).astype(np.float32)
    s[rng.random(s.shape) < 0.3] = 1.5
    s[rng.random(s.shape) < 0.1] = 0.0
    s[rng.random(s.shape) < 0.1] = -0.0
    s[rng.random(s.shape) < 0.1] *= -1
    s[rng.random(s.shape) < 0.02] = np.inf
    s[rng.random(s.shape) < 0.02] = -np.inf
    return s


def check_select(dev, lens, K, sink=0, recent=1, page=16, req=None, seed=0, scores=None, strided=False):
    rng = np.random.default_rng(seed)
    T = len(lens)
    req = list(range(T)) if req is None else req
    most = [max([n for n, r in zip(lens, req) if r == x] + [0]) for x in range(max(req) + 1)]
    table, _ = tables(rng, most, page)
    width = table.shape[1]
    s = rows_of(rng, T, width) if scores is None else scores
    for t, n in enumerate(lens):  # what lies behind the blocks is not looked at
        s[t, -(-max(n, 0) // page):] = np.nan
    d = torch.full((T, width + 3), float("nan"), device=dev)[:, 1:width + 1] if strided else torch.empty((T, width), device=dev)
    d.copy_(torch.from_numpy(s))
    kw = {}
    if strided:
        kw = dict(blocks=torch.full((T, K + 2), -8, dtype=torch.int32, device=dev),
                  table=torch.full((T, K + 1), -8, dtype=torch.int32, device=dev),
                  lengths_out=torch.full((T,), -8, dtype=torch.int32, device=dev))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    blocks, own, out = dsa.dsa_block_select(d, i32(table, dev), i32(lens, dev), K, page_size=page, req_of_token=i32(req, dev),
                                            sink=sink, recent=recent, error_word=err, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    blocks, own, out = blocks.cpu().numpy(), own.cpu().numpy(), out.cpu().numpy()
    for t, n in enumerate(lens):
        n = max(n, 0)
        nb = -(-n // page)
        want = S.select(s[t], nb, K, sink, recent)
        m = len(want)
        assert blocks[t, :m].tolist() == want and (blocks[t, m:K] == -1).all(), t
        assert own[t, :m].tolist() == table[req[t], want].tolist() and (own[t, m:K] == -1).all(), t
        assert out[t] == sum(min(page, n - b * page) for b in want), t
        assert (blocks[t, K:] == -8).all() and (own[t, K:] == -8).all()


@pytest.mark.parametrize("width", [1, 3, 128, 129, 512, 513, 2048, 2049, 8192, 8193, 20000])
@pytest.mark.parametrize("K,sink,recent", [(1, 0, 1), (1, 1, 0), (7, 2, 2), (64, 0, 0), (200, 5, 100)])
def test_select(gpu, width, K, sink, recent):
    lens = [width * 16, width * 16 - 3, 0, 1, width * 8 + 1, min(K, width) * 16, width * 16 - 15]
    check_select(gpu, lens, K, sink, recent, seed=width + K)


@pytest.mark.parametrize("width", [100, 500, 1500, 5000, 12000])
def test_select_ties(gpu, width):
    lens = [width] * 4
    for value in (0.0, 1.0, -np.inf, np.inf):
        check_select(gpu, lens, 33, 2, 3, page=1, scores=np.full((4, width + 2), value, dtype=np.float32))
    s = np.where(np.arange(width + 2) % 3 == 0, 0.0, -0.0).astype(np.float32) * np.ones((4, 1), dtype=np.float32)
    check_select(gpu, lens, 40, 0, 0, page=1, scores=s)
    check_select(gpu, lens, 16384, 0, 16384, page=1)
    s = np.arange(width + 2, dtype=np.float32)[None] * np.float32([[1], [-1], [1e-40], [1e30]])
    check_select(gpu, lens, 50, 1, 1, page=1, scores=s)


def test_select_shared_requests_and_strides(gpu):
    lens = list(range(700, 790)) + list(range(3, 40)) + [0, 0]
    req = [1] * 90 + [0] * 37 + [2, 1]
    check_select(gpu, lens, 9, 1, 2, req=req, strided=True)
    check_select(gpu, lens, 9, 1, 2, req=req, page=1)
    check_select(gpu, [5000, 70], 6, 1, 2, strided=True)


def test_select_bad_entries(gpu):
    s = torch.arange(12, dtype=torch.float32, device=gpu).view(3, 4)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)

    def run(lens, req, cols=4, **kw):
        err.zero_()
        table = i32([[5, 6, 7, 8], [1, 2, -1, 9]], gpu)[:, :cols]
        got = dsa.dsa_block_select(s, table, i32(lens, gpu), 2, page_size=16, req_of_token=i32(req, gpu), error_word=err, **kw)
        return [x.tolist() for x in got], err.item()

    assert run([64, 50, 20], [0, 1, 1]) == ([[[2, 3], [2, 3], [0, 1]], [[7, 8], [-1, 9], [1, 2]], [32, 18, 20]], 0)
    assert run([64, 50, 20], [0, 2, -1]) == ([[[2, 3], [-1, -1], [-1, -1]], [[7, 8], [-1, -1], [-1, -1]], [32, 0, 0]], BAD)
    # more blocks than the table or the scores have: the excess is left out
    assert run([65, 50, 20], [0, 1, 1])[0][0][0] == [2, 3] and err.item() == BAD
    assert run([64, 50, 20], [0, 1, 1], cols=3) == ([[[1, 2], [1, 2], [0, 1]], [[6, 7], [2, -1], [1, 2]], [32, 32, 20]], BAD)
    assert run([2 ** 31 - 1, 5, 5], [0, 1, 1])[0][2] == [32, 5, 5]


def test_select_nan_chooses_as_many(gpu):
    for width in (100, 1000, 10000):
        s = torch.full((2, width), float("nan"), device=gpu)
        s[1] = -s[1]
        blocks, _, lens = dsa.dsa_block_select(s, i32(np.arange(width)[None], gpu), i32([width, width], gpu), 9, page_size=1,
                                               req_of_token=i32([0, 0], gpu))
        b = blocks.cpu().numpy()
        assert (np.diff(b, axis=1) > 0).all() and b.min() >= 0 and b.max() == width - 1 and lens.tolist() == [9, 9]


def test_select_from_a_graph(gpu):
    gen = torch.Generator(device=gpu).manual_seed(3)
    s = torch.randn((50, 900), generator=gen, device=gpu)
    table, lens = i32(np.arange(900)[None], gpu), torch.full((50,), 14400, dtype=torch.int32, device=gpu)
    req = torch.zeros(50, dtype=torch.int32, device=gpu)
    run = lambda: dsa.dsa_block_select(s, table, lens, 20, page_size=16, req_of_token=req, sink=1, recent=2)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    s.copy_(s.flip(1))
    lens -= 100
    want = run()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_binding_refusals(gpu):
    cache, summary = torch.zeros((64, 264), dtype=torch.uint8, device=gpu), torch.zeros((4, 256), dtype=torch.bfloat16, device=gpu)
    table, one = i32([[0, 1]], gpu), i32([1], gpu)
    q, s = torch.zeros((1, 4, 256), dtype=torch.bfloat16, device=gpu), torch.zeros((1, 2), device=gpu)
    pool = dict(cache=cache, kind=FP8, block_table=table, positions=one, lengths=one, summary=summary, page_size=16)
    for name, bad in [("kind", BF16), ("lengths", i32([1, 1], gpu)), ("summary", summary[:, :128]), ("summary", summary.float()),
                      ("req_of_token", i32([0, 0], gpu)), ("block_table", table[:, :0]), ("positions", one.cpu()),
                      ("page_size", 1 << 33)]:
        with pytest.raises(ValueError):
            dsa.dsa_block_pool(**{**pool, name: bad})
    scores = dict(q=q, summary=summary, block_table=table, lengths=one, sm_scale=1.0, page_size=16)
    for name, bad in [("q", q[..., :128]), ("q", q.float()), ("lengths", i32([1, 1], gpu)), ("weights", s), ("out", s[:, :0]),
                      ("out", s.half()), ("block_table", table[0]), ("summary", summary.cpu())]:
        with pytest.raises(ValueError):
            dsa.dsa_block_scores(**{**scores, name: bad})
    with pytest.raises(dsa.DsaError):
        dsa.dsa_block_scores(**{**scores, "sm_scale": -1.0})
    choice = dict(scores=s, block_table=table, lengths=one, K=2, page_size=16)
    for name, bad in [("scores", s.double()), ("K", 0), ("K", 1 << 32), ("blocks", table[:, :1]), ("lengths_out", i32([1, 1], gpu)),
                      ("lengths", one.long())]:
        with pytest.raises(ValueError):
            dsa.dsa_block_select(**{**choice, name: bad})
    for kw in (dict(sink=2), dict(recent=-1), dict(K=16385)):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_block_select(**{**choice, **kw})
    with pytest.raises(dsa.DsaError):  # two tokens, one request, no map
        dsa.dsa_block_select(torch.zeros((2, 2), device=gpu), table, i32([1, 1], gpu), 1, page_size=16)


# ------------------------------------------------------------------------------------ together --
@pytest.mark.parametrize("kind", [BF16, FP8])
def test_serving_steps(gpu, kind):
    """Prefill, decode, an eviction and a request's end: every step's plan, rows, means, scores, choice
    and attention against the definitions, each from the GPU's own state before it."""
    gen = torch.Generator(device=gpu).manual_seed(11)
    R, H, page, width, T, K = 4, 16, 16, 24, 160, 5
    pages = 60
    row = 264 if kind == FP8 else 256
    cache = torch.zeros((pages * page, row), dtype=torch.uint8 if kind == FP8 else torch.bfloat16, device=gpu)
    summary = torch.zeros((pages, 256), dtype=torch.bfloat16, device=gpu)
    lens, held = i32([0] * R, gpu), i32([0] * R, gpu)
    table = torch.full((R, width), -1, dtype=torch.int32, device=gpu)
    free, nfree = torch.randperm(pages, generator=gen, device=gpu).to(torch.int32), i32([pages], gpu)
    mass = torch.zeros((R, width * page), device=gpu)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    wq = (1 + 0.1 * torch.randn(256, generator=gen, device=gpu)).to(torch.bfloat16)
    steps = [[100, 0, 37, 0], [1, 33, 1, 0], [1, 1, 1, 65], "evict", [1, 1, -1, 1], [1, 1, 120, 1]]
    for new in steps:
        if new == "evict":
            dsa.dsa_cache_evict(cache, kind, table, lens, mass, 40, page_size=page, sink=2, recent=8, error_word=err)
            # rows moved: the summaries of what is left are made again
            left = lens.tolist()
            pos = [p for n in left for p in range(n)]
            req = [r for r, n in enumerate(left) for _ in range(n)]
            dsa.dsa_block_pool(cache, kind, table, i32(pos, gpu), lens, summary, page_size=page, req_of_token=i32(req, gpu),
                               error_word=err)
            continue
        want, bits = S.plan(lens.tolist(), new, held.tolist(), table.cpu().numpy().copy(), free.cpu().numpy().copy(),
                            nfree.item(), T, page)
        assert bits == 0
        cu, req, pos, tlen, loc = dsa.dsa_batch_plan(lens, i32(new, gpu), held, table, free, nfree, T, page_size=page,
                                                     error_word=err)
        assert loc.tolist() == want["out_loc"] and tlen.tolist() == want["token_lengths"]
        q = torch.randn((T, H, 256), generator=gen, device=gpu).to(torch.bfloat16)
        k = torch.randn((T, 256), generator=gen, device=gpu).to(torch.bfloat16)
        x = dsa.dsa_qk_norm_rope(q, k, pos, None, 1e-6, cache, kind, loc, q_norm=256, k_norm=256, q_weight=wq, error_word=err)
        dsa.dsa_block_pool(cache, kind, table, pos, lens, summary, page_size=page, req_of_token=req, error_word=err)
        scores = dsa.dsa_block_scores(x, summary, table, tlen, 1 / 16, page_size=page, req_of_token=req, error_word=err)
        blocks, own, own_len = dsa.dsa_block_select(scores, table, tlen, K, page_size=page, req_of_token=req, sink=1, recent=2,
                                                    error_word=err)
        out = dsa.dsa_paged_attn(x, cache, kind, own, own_len, 1 / 16, page_size=page, error_word=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        n = want["cu"][-1]
        assert (out[n:] == 0).all() and (own_len[n:] == 0).all()
        rows, qd, tab = raw(cache), f64(x), table.cpu().numpy()
        means = S.pool(rows, tab, page, req.tolist(), pos.tolist(), lens.tolist())
        sm, sc = f64(summary), scores.cpu().numpy()
        for p, (mean, size, m) in means.items():
            assert (np.abs(sm[p] - mean) <= size * m * 2.0 ** -24 + np.abs(mean) * 2.0 ** -8 * 1.001).all()
        for t in list(range(0, n, 7)) + [n - 1]:
            r, length = req[t].item(), tlen[t].item()
            nb = -(-length // page)
            val, size, terms = S.scores(qd[t], sm, tab[r, :nb], 1 / 16, None)
            assert (np.abs(sc[t, :nb] - val) <= size * 256 * 2.0 ** -23 + terms * (H + 2) * 2.0 ** -24).all()
            picked = S.select(sc[t], nb, K, 1, 2)
            assert blocks[t].tolist() == picked + [-1] * (K - len(picked))
            at = np.concatenate([np.arange(b * page, min((b + 1) * page, length)) for b in picked])
            keys = G.latent_rows(rows, tab[r, at // page].astype(np.int64) * page + at % page)
            o, _, pk, spread = G.softmax_output((qd[t] @ keys.T) / 16, keys)
            # half a bf16 step of the output, and of each weight (spread), beside the sums' 2^-18
            tol = np.abs(o) * 2.0 ** -8 + 2.0 ** -8 * spread * 2 + pk * 2.0 ** -9
            assert (np.abs(f64(out[t]) - o) <= tol + 1e-6).all(), t
        # a weight for the eviction: the newest positions' and a few others'
        mass.copy_(torch.rand(mass.shape, generator=gen, device=gpu))
    live = [p for r in range(R) for p in table[r, :held[r].item()].tolist()] + free[:nfree.item()].tolist()
    assert sorted(live) == list(range(pages))
    assert held.tolist() == [-(-n // page) for n in lens.tolist()]
