"""Dense attention over the paged latent cache and its attention mass on the GPU, against the fp64
definitions (oracle/paged.py).

Tolerances, per element, from the arithmetic the header states (u = 2^-24 fp32, 2^-8 bf16 half steps):
  score    d = 256 * 2^-23 * B + 2^-21 * (|cap| + |bias| + |u|), B = max_j |sm_scale| sum |q k|
           (an fp32 sum of 256 exact products in any order, one step of slack for the tensor core's
           truncation; then a few fp32 operations, the tanh from one exponential); with an FP8 cache
           + 2^-17 |sm_scale| max |q| max_j sum |k| (the query's second e4m3 term: its smallest step
           is 2^-9 where the head's largest component is at least 2^7, half a step is 2^-17 of it)
  lse      d + n 2^-23 + 2^-20 (each exponential 2^-21 relative, their fp32 sum, the logarithm)
  out      2^-8 |out| (its own rounding) + 5 * 2^-8 sqrt(sum (p k)^2) (the weights rounded to bf16:
           independent errors of at most 2^-8 relative each, whose standard deviation is below
           0.58 times that, so five bounds are more than eight deviations)
           + (2 d + n 2^-22 + 2^-20) sum p |k| (scores, fp32 accumulation)
  mass     sum_h w_h (d_h + 2^-20) + (H + 2) 2^-24 |mass_out|
"""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
import oracle as O
from oracle import paged as R
from oracle import projection as P

from _helpers import bf16_dev, f32_of

pytestmark = pytest.mark.gpu

BF16, FP8 = dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED


class Case:
    """Requests of given lengths in scattered pages; host bits and device tensors."""

    def __init__(self, dev, kind, lens, H, page=64, seed=0, T=None, req=None, spread=0.5, q_scale=1.0, direct=False):
        rng = np.random.default_rng(seed)
        self.kind, self.H, self.page, self.dev, self.direct = kind, H, page, dev, direct
        self.lens = np.asarray(lens, dtype=np.int32)
        self.req = None if req is None else np.asarray(req, dtype=np.int32)
        T = len(lens)
        nreq = T if req is None else int(max(req)) + 1
        need = np.zeros(nreq, dtype=np.int64)
        for t in range(T):
            r = t if req is None else req[t]
            need[r] = max(need[r], (max(int(self.lens[t]), 0) + page - 1) // page)
        pages = int(need.sum()) + 3
        perm = rng.permutation(pages)
        self.bt = np.full((nreq, max(int(need.max()), 1) + 1), -1, dtype=np.int32)
        at = 0
        for r in range(nreq):
            self.bt[r, :need[r]] = perm[at:at + need[r]]
            at += need[r]
        slots = max(int(self.lens.max()), 1) + 5 if direct else pages * page
        rows = rng.standard_normal((slots, 256)) * np.exp(spread * rng.standard_normal((slots, 1)))
        bits = P.f64_to_bf16(rows)
        self.cache = bits if kind == BF16 else O.quant_k_cache(bits, num_slots=slots)
        self.q = P.f64_to_bf16(q_scale * rng.standard_normal((T, H, 256)))
        self.sm_scale = 1 / 16
        if direct:
            self.bt = None

    def cache_dev(self):
        return bf16_dev(self.cache, self.dev) if self.kind == BF16 else torch.from_numpy(self.cache).to(self.dev)

    def table(self):
        return None if self.bt is None else torch.from_numpy(self.bt).to(self.dev)

    def args(self):
        return (bf16_dev(self.q, self.dev), self.cache_dev(), self.kind, self.table(),
                torch.from_numpy(self.lens).to(self.dev), self.sm_scale)

    def opts(self, **kw):
        o = {"page_size": 0 if self.direct else self.page, **kw}
        if self.req is not None:
            o["req_of_token"] = torch.from_numpy(self.req).to(self.dev)
        return o

    def reference(self, t, starts=None, cap=0.0, slopes=None, qpos=None, kpos=None):
        r = t if self.req is None else int(self.req[t])
        b = int(self.lens[t])
        a = 0 if starts is None else int(starts[t])
        qp = b - 1 if qpos is None else int(qpos[t])
        u, k, pos, bound = R.scores(P.bf16_to_f64(self.q[t]), self.cache, self.bt, self.page, r, a, b, self.sm_scale,
                                    cap, slopes, qp, kpos)
        bias = 0.0
        if slopes is not None and len(pos):
            kp = pos if kpos is None else kpos[r][pos]
            bias = np.abs(slopes).max() * np.abs(qp - kp).max()
        umax = np.abs(u).max(axis=1) if u.shape[1] else np.zeros(self.H)
        d = 256 * 2.0 ** -23 * bound + 2.0 ** -21 * (abs(cap) + bias + umax)
        if self.kind == FP8 and len(pos):
            d = d + 2.0 ** -17 * abs(self.sm_scale) * np.abs(P.bf16_to_f64(self.q[t])).max(axis=1) * np.abs(k).sum(1).max()
        return u, k, pos, d


def dev_t(x, dev):
    return None if x is None else torch.from_numpy(np.asarray(x)).to(dev)


def run_and_check(c, starts=None, cap=0.0, slopes=None, qpos=None, kpos=None, want_err=0, **kw):
    dev = c.dev
    opts = c.opts(starts=dev_t(starts, dev), logit_cap=cap, slopes=dev_t(slopes, dev), q_positions=dev_t(qpos, dev),
                  key_positions=dev_t(kpos, dev))
    T = len(c.lens)
    lse = torch.full((T, c.H), float("nan"), device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = dsa.dsa_paged_attn(*c.args(), lse=lse, error_word=err, **opts, **kw)
    torch.cuda.synchronize()
    assert err.item() == want_err
    got, glse = f32_of(out).astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    for t in range(T):
        u, k, pos, d = c.reference(t, starts, cap, slopes, qpos, kpos)
        ref, rl, absum, l2 = R.softmax_output(u, k)
        n = len(pos)
        if n == 0:
            assert (got[t] == 0).all() and np.isneginf(glse[t]).all(), t
            continue
        e = np.abs(glse[t] - rl)
        assert (e <= d + n * 2.0 ** -23 + 2.0 ** -20).all(), (t, e.max(), d.max())
        tol = 2.0 ** -8 * np.abs(ref) + 5 * 2.0 ** -8 * l2 + (2 * d[:, None] + n * 2.0 ** -22 + 2.0 ** -20) * absum
        e = np.abs(got[t] - ref)
        assert (e <= tol).all(), (t, n, np.unravel_index(np.argmax(e - tol), e.shape), e.max())
        # and as a whole: rounding errors do not line up, a wrong row or a lost part does
        assert np.linalg.norm(e) <= 2.0 ** -7 * np.linalg.norm(ref) + 2.0 ** -7 * np.linalg.norm(l2), t
    return out, lse, opts


def check_mass(c, lse, opts, starts=None, cap=0.0, slopes=None, qpos=None, kpos=None, width=None):
    dev = c.dev
    rng = np.random.default_rng(5)
    nreq = len(c.lens) if c.req is None else int(c.req.max()) + 1
    if c.bt is not None:
        nreq = c.bt.shape[0]
    S = max(int(c.lens.max()), 1) + 7 if width is None else width
    m0 = rng.random((nreq, S)).astype(np.float32)
    mass = torch.from_numpy(m0).to(dev)
    before = torch.full_like(mass, -5.0)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = dsa.dsa_paged_attn_mass(*c.args(), lse, mass, mass_out=before, error_word=err, **opts)
    inplace = dsa.dsa_paged_attn_mass(*c.args(), lse, mass, **opts)
    torch.cuda.synchronize()
    assert err.item() == 0
    got, got2 = out.cpu().numpy().astype(np.float64), inplace.cpu().numpy().astype(np.float64)
    ref, tol = m0.astype(np.float64), np.zeros(m0.shape)
    inside = np.zeros(m0.shape, dtype=bool)
    gl = lse.cpu().numpy().astype(np.float64)
    for t in range(len(c.lens)):
        r = t if c.req is None else int(c.req[t])
        a = 0 if starts is None else max(int(starts[t]), 0)
        inside[r, a:max(int(c.lens[t]), a)] = True
        u, k, pos, d = c.reference(t, starts, cap, slopes, qpos, kpos)
        if len(pos):
            w = np.exp(u - gl[t][:, None])
            ref[r, pos] += w.sum(axis=0)
            tol[r, pos] = (w * (d[:, None] + 2.0 ** -20)).sum(axis=0)
    tol += (c.H + 2) * 2.0 ** -24 * np.abs(ref)
    assert (np.abs(got - ref)[inside] <= tol[inside]).all(), np.abs(got - ref)[inside].max()
    assert (got[~inside] == -5.0).all()
    assert (got2[inside] == got[inside]).all() and (got2[~inside] == m0[~inside]).all()


RAGGED = [0, 1, 2, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("page", [1, 3, 16, 64, 128, 200])
def test_ragged_lengths_and_page_sizes(gpu, kind, page):
    c = Case(gpu, kind, RAGGED, 64, page, seed=page)
    out, lse, opts = run_and_check(c)
    check_mass(c, lse, opts)


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("H", [1, 3, 8, 16, 17, 32, 33, 64, 65, 100, 128])
def test_heads(gpu, kind, H):
    c = Case(gpu, kind, [5, 400, 1], H, seed=H)
    out, lse, opts = run_and_check(c)
    check_mass(c, lse, opts)


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("lens", [[1], [64], [2049], [20000], [3, 9000], [700] * 40, [130] * 200])
def test_splits(gpu, kind, lens):
    """One token over the whole device, many tokens per CTA, and between: every split and join."""
    c = Case(gpu, kind, lens, 16, seed=len(lens))
    out, lse, opts = run_and_check(c)
    check_mass(c, lse, opts)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_full_heads_split(gpu, kind):
    c = Case(gpu, kind, [5000, 1, 7777], 64, seed=4)
    run_and_check(c)


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("cap,bias,doc", [(30.0, False, False), (0.0, True, False), (0.0, False, True), (5.0, True, True)])
def test_cap_bias_documents(gpu, kind, cap, bias, doc):
    H = 24
    lens = [0, 1, 129, 700, 2500]
    c = Case(gpu, kind, lens, H, seed=11, q_scale=4.0)
    slopes = np.exp2(-8.0 * (np.arange(H) + 1) / H).astype(np.float32) if bias else None
    starts = np.array([0, 1, -4, 333, 1281], dtype=np.int32) if doc else None
    out, lse, opts = run_and_check(c, starts=starts, cap=cap, slopes=slopes)
    check_mass(c, lse, opts, starts=starts, cap=cap, slopes=slopes)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_positions_after_an_eviction(gpu, kind):
    """Key positions out of order, and query positions other than the last."""
    rng = np.random.default_rng(3)
    lens = [50, 600]
    c = Case(gpu, kind, lens, 8, seed=13)
    kpos = rng.permutation(2 * 700).reshape(2, 700).astype(np.int32)
    qpos = np.array([1400, 700], dtype=np.int32)
    slopes = np.linspace(0.01, 0.2, 8).astype(np.float32)
    out, lse, opts = run_and_check(c, slopes=slopes, qpos=qpos, kpos=kpos)
    check_mass(c, lse, opts, slopes=slopes, qpos=qpos, kpos=kpos)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_direct_slots_and_shared_request(gpu, kind):
    c = Case(gpu, kind, [900, 1, 0, 257], 64, seed=2, direct=True)
    run_and_check(c)
    c = Case(gpu, kind, [300, 299, 298, 40], 64, seed=2, req=[1, 1, 1, 0])
    run_and_check(c)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_rows_outside_the_range_may_hold_nan(gpu, kind):
    lens = [1, 130, 700]
    starts = np.array([0, 60, 411], dtype=np.int32)
    c = Case(gpu, kind, lens, 64, seed=21)
    used = np.zeros(c.cache.shape[0], dtype=bool)
    for r, n in enumerate(lens):
        used[R.slots_of(c.bt, c.page, c.cache.shape[0], r, np.arange(starts[r], n))] = True
    c.cache[~used] = 0x7FC0 if kind == BF16 else 0x7F
    if kind == FP8:
        c.cache[~used, 256:] = 0xFF  # NaN scales
    out, lse, opts = run_and_check(c, starts=starts)
    check_mass(c, lse, opts, starts=starts)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_bad_pages_requests_and_lengths_are_masked(gpu, kind):
    lens = [300, 500, 64, 2000]
    c = Case(gpu, kind, lens, 32, seed=8)
    c.bt[0, 1] = -7                    # a negative page in the middle
    c.bt[1, 0] = c.cache.shape[0]      # a page past the pool
    c.bt[2, 0] = 2 ** 31 - 1
    c.lens[3] = c.bt.shape[1] * 64 + 999   # past the table: its last column is -1 as well
    run_and_check(c, want_err=dsa.DEVERR_INDEX_OUT_OF_RANGE)
    c = Case(gpu, kind, [40, 50], 32, seed=8)
    c.req = np.array([7, -1], dtype=np.int32)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    lse = torch.zeros((2, 32), device=gpu)
    out = dsa.dsa_paged_attn(*c.args(), lse=lse, error_word=err, **c.opts())
    torch.cuda.synchronize()
    assert err.item() == dsa.DEVERR_INDEX_OUT_OF_RANGE and (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_scales_and_large_scores(gpu, kind):
    """sm_scale 0 and negative; scores in the hundreds, growing along the range (the running
    maximum is raised many times), and falling."""
    c = Case(gpu, kind, [1, 200, 1500], 64, seed=6)
    for s in (0.0, -0.25, 0.5):
        c.sm_scale = s
        run_and_check(c)
    c.sm_scale = 1 / 16
    rng = np.random.default_rng(1)
    base = rng.standard_normal(256)
    for sign in (1, -1):
        n = 1500
        ramp = np.linspace(0.1, 20.0, n)[::sign]
        rows = P.f64_to_bf16(ramp[:, None] * base[None, :] + 0.1 * rng.standard_normal((n, 256)))
        slot = R.slots_of(c.bt, 64, c.cache.shape[0], 2, np.arange(n))
        c.cache[slot] = rows if kind == BF16 else O.quant_k_cache(rows, num_slots=n)
        c.q[2, :] = P.f64_to_bf16(np.linspace(-2, 2, 64)[:, None] * base[None, :])
        run_and_check(c)


def test_fp8_tile_scales_far_apart(gpu):
    """The two tiles of a row, and rows among themselves, 2^40 apart: each output column keeps its
    precision whatever the other's scale."""
    c = Case(gpu, FP8, [3, 400], 64, seed=31)
    rng = np.random.default_rng(2)
    sc = np.exp2(rng.integers(-40, 1, size=(c.cache.shape[0], 2))).astype(np.float32)
    c.cache[:, 256:] = sc.view(np.uint8).reshape(-1, 8)
    c.sm_scale = 1e-3
    run_and_check(c)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_strided_tensors(gpu, kind):
    c = Case(gpu, kind, [70, 513, 128], 40, seed=17)
    q, cache, k, bt, lens, s = c.args()
    wide = torch.zeros((40, 3, 264), dtype=torch.bfloat16, device=gpu)
    wide[:, :, :256] = q.transpose(0, 1)
    qs = wide.transpose(0, 1)[:, :, :256]
    bts = torch.full((3, bt.shape[1] + 5), -9, dtype=torch.int32, device=gpu)
    bts[:, :bt.shape[1]] = bt
    out_w = torch.full((40, 3, 272), 7.0, dtype=torch.bfloat16, device=gpu)
    ref = dsa.dsa_paged_attn(q, cache, k, bt, lens, s, page_size=64)
    got = dsa.dsa_paged_attn(qs, cache, k, bts[:, :bt.shape[1]], lens, s, page_size=64,
                             out=out_w.transpose(0, 1)[:, :, :256])
    torch.cuda.synchronize()
    assert torch.equal(got, ref) and (out_w[:, :, 256:] == 7.0).all()


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_repeats_streams_and_graphs(gpu, kind):
    """Bit-identical repeats, two streams at once, and two captured graphs replayed in turn and
    with changed lengths."""
    c = Case(gpu, kind, [4000, 37, 900], 64, seed=19)
    d = Case(gpu, kind, [100, 6000], 64, seed=20)
    ca, da = c.args(), d.args()
    ref_c = dsa.dsa_paged_attn(*ca, page_size=64)
    ref_d = dsa.dsa_paged_attn(*da, page_size=64)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            o1 = dsa.dsa_paged_attn(*ca, page_size=64)
        with torch.cuda.stream(s2):
            o2 = dsa.dsa_paged_attn(*da, page_size=64)
        torch.cuda.synchronize()
        assert torch.equal(o1, ref_c) and torch.equal(o2, ref_d)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = dsa.dsa_paged_attn(*ca, page_size=64)
    with torch.cuda.graph(g2):
        o2 = dsa.dsa_paged_attn(*da, page_size=64)
    for _ in range(3):
        o1.zero_(), o2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, ref_c) and torch.equal(o2, ref_d)
    ca[4].copy_(torch.tensor([200, 37, 0], dtype=torch.int32))
    ref = dsa.dsa_paged_attn(*ca, page_size=64)
    g1.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, ref)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_tiles_without_a_valid_key(gpu, kind):
    """Whole tiles of bad pages before, between and after valid ones, scores far from zero."""
    c = Case(gpu, kind, [1200, 5000], 24, seed=37, q_scale=20.0)
    c.bt[0, 0:4] = -1
    c.bt[0, 8:11] = -5
    c.bt[1, 2:40] = -1
    c.bt[1, 70:79] = c.cache.shape[0]
    run_and_check(c, want_err=dsa.DEVERR_INDEX_OUT_OF_RANGE)


def test_mass_refuses_repeated_and_unordered_requests(gpu):
    c = Case(gpu, BF16, [20, 30, 40, 50], 8, seed=23, req=[1, 3, 1, 3])
    lse = torch.zeros((4, 8), device=gpu)
    dsa.dsa_paged_attn(*c.args(), lse=lse, **c.opts())
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    mass = torch.zeros((4, 64), device=gpu)
    dsa.dsa_paged_attn_mass(*c.args(), lse, mass, error_word=err, **c.opts())
    torch.cuda.synchronize()
    assert err.item() == dsa.DEVERR_REQUEST_ORDER
    m = mass.cpu().numpy()
    assert (m[[0, 2]] == 0).all()
    # requests 1 and 3 from tokens 0 and 1 alone: eight heads' weights sum to eight
    assert np.allclose(m[1].sum(), 8, rtol=1e-4) and (m[1, 20:] == 0).all()
    assert np.allclose(m[3].sum(), 8, rtol=1e-4) and (m[3, 30:] == 0).all()


def test_mass_with_sparse_requests(gpu):
    c = Case(gpu, FP8, [20, 0, 400], 16, seed=29, req=[1, 2, 5])
    out, lse, opts = run_and_check(c)
    check_mass(c, lse, opts)


def test_empty_batch(gpu):
    q = torch.empty((0, 64, 256), dtype=torch.bfloat16, device=gpu)
    cache = torch.zeros((64, 256), dtype=torch.bfloat16, device=gpu)
    bt = torch.zeros((1, 1), dtype=torch.int32, device=gpu)
    out = dsa.dsa_paged_attn(q, cache, BF16, bt, torch.empty(0, dtype=torch.int32, device=gpu), 1.0, page_size=64)
    assert tuple(out.shape) == (0, 64, 256)


def test_slots_past_32_bits_of_bytes(gpu):
    """Rows more than 2^32 bytes into the cache."""
    slots = (1 << 32) // 512 + 640
    cache = torch.zeros((slots, 256), dtype=torch.bfloat16, device=gpu)
    small = Case(gpu, BF16, [256], 64, seed=41)
    pages = small.bt[0, :4].copy()
    far = slots // 64 - 1 - np.arange(4)
    src = small.cache_dev()
    for a, b in zip(pages, far):
        cache[b * 64:(b + 1) * 64] = src[a * 64:(a + 1) * 64]
    q, _, k, bt, lens, s = small.args()
    ref = dsa.dsa_paged_attn(q, src, k, bt, lens, s, page_size=64)
    bt2 = bt.clone()
    bt2[0, :4] = torch.from_numpy(far.astype(np.int32))
    got = dsa.dsa_paged_attn(q, cache, k, bt2, lens, s, page_size=64)
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("n,H,top", [(257, 1, 3), (300, 8, 400), (300, 65, 300), (1500, 2, 140)])
def test_many_tokens(gpu, kind, n, H, top):
    """More rows than one warp plans, far more than CTAs, empty ones among them."""
    lens = np.random.default_rng(n + H).integers(0, top + 1, n)
    lens[lens % 5 == 0] = 0
    c = Case(gpu, kind, lens, H, 16, seed=n)
    out, lse, opts = run_and_check(c)
    check_mass(c, lse, opts)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_many_tokens_of_one_request(gpu, kind):
    """A prompt's last tokens, each attending to all before it."""
    c = Case(gpu, kind, np.arange(1, 301), 4, 64, seed=43, req=[0] * 300)
    run_and_check(c)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_mass_order_among_many_tokens(gpu, kind):
    """Requests out of order and repeated, in a batch that the whole block plans: the mass holds what
    the tokens in order give, the others add nothing."""
    n, H = 400, 8
    rng = np.random.default_rng(47)
    req = np.arange(n)
    back = np.sort(rng.choice(np.arange(1, n), 60, replace=False))
    req[back] = [rng.integers(0, i) for i in back]
    c = Case(gpu, kind, rng.integers(1, 300, n), H, 16, seed=53, req=req)
    q, cache, k, bt, lens, s = c.args()
    opts = c.opts()
    lse = torch.zeros((n, H), device=gpu)
    dsa.dsa_paged_attn(*c.args(), lse=lse, **opts)
    good = np.zeros(n, dtype=bool)
    top = -1
    for i in range(n):
        good[i] = req[i] > top
        top = max(top, req[i])
    assert not good[back].any() and good.sum() == n - 60
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    mass = torch.zeros((c.bt.shape[0], 310), device=gpu)
    dsa.dsa_paged_attn_mass(*c.args(), lse, mass, error_word=err, **opts)
    torch.cuda.synchronize()
    assert err.item() == dsa.DEVERR_REQUEST_ORDER
    got = mass.cpu().numpy().astype(np.float64)
    gl = lse.cpu().numpy().astype(np.float64)
    ref, tol = np.zeros(got.shape), np.zeros(got.shape)
    for t in np.flatnonzero(good):
        u, _, pos, d = c.reference(t)
        w = np.exp(u - gl[t][:, None])
        ref[req[t], pos] = w.sum(axis=0)
        tol[req[t], pos] = (w * (d[:, None] + 2.0 ** -20)).sum(axis=0)
    tol += (H + 2) * 2.0 ** -24 * np.abs(ref)
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("page", [33, 65, 129, 255])
@pytest.mark.parametrize("start", [0, 1, 97])
def test_fp8_rows_from_odd_slots(gpu, page, start):
    """Pages of an odd number of rows: runs of rows begin at odd and at even slots, where an FP8 row
    (264 bytes) starts on 8 and on 16 bytes."""
    c = Case(gpu, FP8, [700, 333, 2000], 16, page, seed=page + start)
    # pages that follow one another from an odd and from an even one: whole tiles of adjacent rows
    c.bt[2, :6] = np.arange(3, 9)
    c.bt[1, :2] = [2, 3]
    starts = np.array([start, start, start], dtype=np.int32)
    out, lse, opts = run_and_check(c, starts=starts)
    check_mass(c, lse, opts, starts=starts)


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_mass_streams_and_graphs(gpu, kind):
    """Two streams at once, and two captured graphs replayed in turn."""
    c = Case(gpu, kind, [3000, 45], 64, seed=59)
    d = Case(gpu, kind, [129, 2500], 33, seed=61)
    calls = []
    for x in (c, d):
        lse = torch.zeros((2, x.H), device=gpu)
        a = x.args()
        dsa.dsa_paged_attn(*a, lse=lse, page_size=64)
        mass = torch.rand((2, 3010), device=gpu)
        to = torch.zeros_like(mass)
        calls.append((a, lse, mass, to))
    def go(i):
        a, lse, mass, to = calls[i]
        dsa.dsa_paged_attn_mass(*a, lse, mass, mass_out=to, page_size=64)
    go(0), go(1)
    torch.cuda.synchronize()
    ref = [calls[0][3].clone(), calls[1][3].clone()]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            go(i)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for call in (go, lambda i: graphs[i].replay()):
        for _ in range(3):
            calls[0][3].zero_(), calls[1][3].zero_()
            torch.cuda.synchronize()
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    call(i)
            torch.cuda.synchronize()
            assert torch.equal(calls[0][3], ref[0]) and torch.equal(calls[1][3], ref[1])


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_mass_of_bad_pages(gpu, kind, cap):
    """Positions of bad pages, a whole request of them (its lse is -inf) among them: they add nothing
    and are copied."""
    lens = [300, 200, 64]
    c = Case(gpu, kind, lens, 32, seed=67)
    c.bt[0, 1] = -7
    c.bt[1, :] = -1
    c.bt[2, 0] = c.cache.shape[0]
    lse = torch.zeros((3, 32), device=gpu)
    dsa.dsa_paged_attn(*c.args(), lse=lse, logit_cap=cap, **c.opts())
    m0 = np.random.default_rng(71).random((3, 310)).astype(np.float32)
    mass = torch.from_numpy(m0).to(gpu)
    to = torch.full_like(mass, -5.0)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    dsa.dsa_paged_attn_mass(*c.args(), lse, mass, mass_out=to, error_word=err, logit_cap=cap, **c.opts())
    torch.cuda.synchronize()
    assert err.item() == dsa.DEVERR_INDEX_OUT_OF_RANGE
    got, gl = to.cpu().numpy(), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(gl[0]).all() and np.isneginf(gl[1:]).all()
    assert (got[0, 64:128] == m0[0, 64:128]).all()
    assert (got[1, :200] == m0[1, :200]).all() and (got[2, :64] == m0[2, :64]).all()
    assert (got[0, 300:] == -5).all() and (got[1, 200:] == -5).all() and (got[2, 64:] == -5).all()
    u, _, pos, d = c.reference(0, cap=cap)
    w = np.exp(u - gl[0][:, None])
    ref = m0[0].astype(np.float64)
    ref[pos] += w.sum(axis=0)
    tol = (c.H + 2) * 2.0 ** -24 * np.abs(ref)
    tol[pos] += (w * (d[:, None] + 2.0 ** -20)).sum(axis=0)
    assert (np.abs(got[0] - ref) <= tol)[:300].all()


def test_tables_without_columns_are_refused(gpu):
    """An empty tensor has no address: it must not pass for no table, which means direct slots."""
    c = Case(gpu, BF16, [40, 50], 8, seed=73)
    q, cache, kind, bt, lens, s = c.args()
    none = torch.empty((2, 0), dtype=torch.int32, device=gpu)
    lse = torch.zeros((2, 8), device=gpu)
    mass = torch.zeros((2, 64), device=gpu)
    with pytest.raises(ValueError, match="block_table"):
        dsa.dsa_paged_attn(q, cache, kind, none, lens, s, page_size=64)
    with pytest.raises(ValueError, match="block_table"):
        dsa.dsa_paged_attn_mass(q, cache, kind, none, lens, s, lse, mass, page_size=64)
    with pytest.raises(ValueError, match="key_positions"):
        dsa.dsa_paged_attn(q, cache, kind, bt, lens, s, page_size=64, slopes=torch.ones(8, device=gpu),
                           key_positions=none)
    with pytest.raises(ValueError, match="block_table"):
        dsa.dsa_cache_evict(cache, kind, none, lens, mass, 8, page_size=64)
    # a batch without tokens may bring one
    assert dsa.dsa_paged_attn(q[:0], cache, kind, none[:0], lens[:0], s, page_size=64).shape[0] == 0
