"""Tokens' places in their sequences beside their positions in the cache: what the batch plan counts
(``seen``, ``token_positions``, ``key_positions``), and that rotation and distance bias are those of the
sequence after evictions."""
import ctypes

import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from oracle import paged as G
from oracle import steps as S

BF16, FP8 = dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED
BAD = dsa.DEVERR_INDEX_OUT_OF_RANGE
NAMES = ("cu", "req", "positions", "token_lengths", "out_loc", "token_positions")


def i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


def pages(n, page):
    return -(-max(int(n), 0) // page)


def build(rng, held, width, spare):
    perm = rng.permutation(int(sum(held)) + spare).astype(np.int32)
    table = np.full((len(held), width), -7, dtype=np.int32)
    at = 0
    for r, c in enumerate(held):
        table[r, :c] = perm[at:at + c]
        at += c
    stack = np.full(len(perm), -9, dtype=np.int32)
    stack[:spare] = perm[at:]
    return table, stack


def check(dev, lens, new, seen, T, page=16, width=40, kp=None, inplace=True, want_err=0, with_seen=True, spare=None):
    rng = np.random.default_rng(len(lens) + T)
    held = [pages(n, page) for n in lens]
    spare = sum(pages(n, page) + 1 for n in new) if spare is None else spare
    table, stack = build(rng, held, width, spare)
    d_table, d_stack = torch.empty((len(lens), width), dtype=torch.int32, device=dev), i32(stack, dev)
    d_table.copy_(i32(table.reshape(len(lens), width), dev))
    kpos = rng.integers(0, 1000, (len(lens), width * page if kp is None else kp)).astype(np.int32)
    wide = torch.full((len(lens), kpos.shape[1] + 3), -5, dtype=torch.int32, device=dev)
    d_kpos = wide[:, :kpos.shape[1]]
    d_kpos.copy_(i32(kpos, dev))
    d_seen = i32(seen, dev)
    kw = {"seen": d_seen} if with_seen else {"token_positions": torch.full((T,), -8, dtype=torch.int32, device=dev)}
    if not inplace:
        kw["seen_out"] = torch.full_like(d_seen, -3)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = dsa.dsa_batch_plan(i32(lens, dev), i32(new, dev), i32(held, dev), d_table, d_stack, i32([spare], dev), T,
                             page_size=page, error_word=err, key_positions=d_kpos, **kw)
    torch.cuda.synchronize()
    want, bits = S.plan(lens, new, held, table, stack, spare, T, page, seen if with_seen else None, kpos)
    assert err.item() == bits == want_err
    assert len(got) == 6
    for name, t in zip(NAMES, got):
        assert t.cpu().tolist() == want[name], name
    assert np.array_equal(d_table.cpu().numpy(), table)
    assert np.array_equal(d_kpos.cpu().numpy(), kpos) and (wide[:, kpos.shape[1]:] == -5).all()
    if with_seen:
        assert (d_seen if inplace else kw["seen_out"]).tolist() == want["seen"]
    if not inplace or not with_seen:
        assert d_seen.tolist() == list(seen)


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("R,most,T", [(1, 1, 1), (5, 30, 90), (300, 9, 1500), (300, 120, 20000), (1025, 3, 2500),
                                      (2100, 12, 16385), (2100, 15, 17000)])
def test_places(gpu, R, most, T, inplace):
    """One block, the cluster, tokens by a launch of their own, several passes over the requests."""
    rng = np.random.default_rng(R + most)
    lens = rng.integers(0, 200, R)
    new = rng.integers(-1, most + 1, R)
    new[0] = most
    while new[new > 0].sum() > T:
        new = new // 2
    check(gpu, lens.tolist(), new.tolist(), (lens + rng.integers(0, 5000, R)).tolist(), T, inplace=inplace)


@pytest.mark.gpu
def test_places_without_a_count(gpu):
    check(gpu, [5, 0, 700], [3, 40, 1], [0, 0, 0], 50, width=60, with_seen=False)


@pytest.mark.gpu
def test_refusals_and_ends(gpu):
    top = 2 ** 31 - 1
    check(gpu, [5, 5, 5], [2, 2, 2], [top - 2, top - 1, top], 8, want_err=BAD)  # the second and third are refused
    check(gpu, [5, 5, 5], [0, -1, 0], [top, top, -4], 8)  # none adds a token; an end starts anew
    check(gpu, [30, 29, 31, 40], [1, 3, 1, 0], [100, 100, 100, 100], 8, kp=31, want_err=BAD)  # 31 entries
    check(gpu, [5, 5], [1, 1], [9, 9], 1, want_err=dsa.DEVERR_TOKEN_CAPACITY)  # a refused request's count stays
    check(gpu, [15, 16], [1, 1], [90, 95], 4, spare=0, want_err=dsa.DEVERR_OUT_OF_PAGES)
    check(gpu, [], [], [], 4)


@pytest.mark.gpu
def test_binding(gpu):
    ok = dict(lengths=i32([1, 1], gpu), new_tokens=i32([1, 1], gpu), held=i32([1, 1], gpu), block_table=i32([[0], [1]], gpu),
              free_pages=i32([2], gpu), num_free=i32([1], gpu), tokens=2, page_size=16)
    assert len(dsa.dsa_batch_plan(**ok)) == 5
    for name, bad in [("seen", i32([1], gpu)), ("seen", i32([1, 1], gpu).long()), ("seen_out", i32([1, 1], gpu)),
                      ("token_positions", i32([0], gpu)), ("key_positions", i32([[0] * 9], gpu)),
                      ("key_positions", i32([0, 0], gpu)), ("key_positions", torch.zeros((2, 9), device=gpu))]:
        with pytest.raises(ValueError):
            dsa.dsa_batch_plan(**ok, **{name: bad})


PTR = 0x10000


@pytest.mark.parametrize("fields", [
    {"seen": PTR}, {"seen": PTR, "seen_out": PTR + 2}, {"seen": PTR + 1, "seen_out": PTR}, {"token_positions": PTR + 2},
    {"key_positions": PTR, "kp_stride": 8, "kp_width": 9}, {"key_positions": PTR, "kp_stride": 8, "kp_width": -1},
    {"key_positions": PTR + 2, "kp_stride": 8, "kp_width": 8}])
def test_refusals_of_the_call(dsa_lib, fields):
    a = dsa.DsaPlanArgs()
    for name in ("lengths", "new_tokens", "held", "block_table", "free_pages", "num_free", "lengths_out", "held_out",
                 "num_free_out", "cu_tokens", "req_of_token", "positions", "token_lengths", "out_loc"):
        setattr(a, name, PTR)
    a.num_requests, a.bt_stride, a.page_size, a.max_pages, a.free_capacity, a.T = 4, 10, 64, 10, 100, 8
    for name, value in fields.items():
        setattr(a, name, value)
    assert dsa_lib.dsa_batch_plan(ctypes.byref(a), None) == 1


class Sequences:
    """Requests that grow and shrink: the GPU's state, and each request's tokens as the host knows them."""

    def __init__(self, dev, kind, nope, rope, R=3, page=16, width=12, pool=40, T=96):
        self.dev, self.kind, self.nope, self.rope, self.page, self.R, self.T = dev, kind, nope, rope, page, R, T
        self.gen = torch.Generator(device=dev).manual_seed(nope + kind)
        row = nope + rope if kind == BF16 else nope + nope // 32 + 2 * rope
        self.cache = torch.zeros((pool * page, row), dtype=torch.bfloat16 if kind == BF16 else torch.uint8, device=dev)
        self.lens, self.held, self.seen = (i32([0] * R, dev) for _ in range(3))
        self.table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
        self.free, self.nfree = torch.randperm(pool, generator=self.gen, device=dev).to(torch.int32), i32([pool], dev)
        self.kpos = torch.full((R, width * page), -1, dtype=torch.int32, device=dev)
        self.mass = torch.zeros((R, width * page), device=dev)
        a = torch.rand((400, max(rope // 2, 1)), generator=self.gen, device=dev, dtype=torch.float64) * 6.3
        self.angles = torch.cat([a.cos(), a.sin()], dim=1).float() if rope else None
        self.keys = [[] for _ in range(R)]  # the bf16 key of each token that the request was given
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)

    def grow(self, new):
        R, T = self.R, self.T
        q = torch.randn((T, 16, self.nope + self.rope), generator=self.gen, device=self.dev).to(torch.bfloat16)
        k = torch.randn((T, self.nope + self.rope), generator=self.gen, device=self.dev).to(torch.bfloat16)
        cu, req, pos, tlen, loc, place = dsa.dsa_batch_plan(
            self.lens, i32(new, self.dev), self.held, self.table, self.free, self.nfree, T, page_size=self.page,
            error_word=self.err, seen=self.seen, key_positions=self.kpos)
        x = dsa.dsa_qk_norm_rope(q, k, place, self.angles, 1e-6, self.cache, self.kind, loc, d_nope=self.nope, d_rope=self.rope,
                                 k_norm=self.nope, error_word=self.err)
        torch.cuda.synchronize()
        assert self.err.item() == 0
        for r in range(R):
            if new[r] < 0:
                self.keys[r] = []
        for t in range(cu[-1].item()):
            r = req[t].item()
            assert place[t].item() == len(self.keys[r])  # the token's place in its sequence
            self.keys[r].append(k[t].clone())
        return x, q, req, pos, tlen, place

    def evict(self, budget):
        self.mass.copy_(torch.rand(self.mass.shape, generator=self.gen, device=self.dev))
        dsa.dsa_cache_evict(self.cache, self.kind, self.table, self.lens, self.mass, budget, page_size=self.page, sink=2, recent=0,
                            positions=self.kpos, d_nope=self.nope, d_rope=self.rope, error_word=self.err)

    def check_rows(self):
        """Every cached row is its token's, normalised, and turned by the angle of its place."""
        table, kpos = self.table.cpu().numpy(), self.kpos.cpu().numpy()
        n = 0
        for r, length in enumerate(self.lens.tolist()):
            at = kpos[r, :length]
            assert len(set(at.tolist())) == length and (length == 0 or at.max() < len(self.keys[r]))
            if not length:
                continue
            x = torch.stack([self.keys[r][j] for j in at])
            j = np.arange(length)
            slots = torch.from_numpy(table[r, j // self.page].astype(np.int64) * self.page + j % self.page).to(self.dev)
            want = torch.zeros((length, self.cache.shape[1]), dtype=self.cache.dtype, device=self.dev)
            dsa.dsa_qk_norm_rope(k=x, positions=i32(at, self.dev), cos_sin=self.angles, eps=1e-6, cache=want, kind=self.kind,
                                 d_nope=self.nope, d_rope=self.rope, k_norm=self.nope)
            assert torch.equal(self.cache[slots], want), r
            if self.rope:  # and that is the definition's rotation
                ang = self.angles.cpu().double().numpy()[at]
                y, size = S.norm_rope(x.cpu().double().numpy(), self.nope, None, 1e-6, ang, False)
                tail = want[:, -2 * self.rope:].contiguous().view(torch.bfloat16) if self.kind == FP8 else want[:, -self.rope:]
                off = np.abs(tail.cpu().double().numpy() - y[:, -self.rope:])
                assert (off <= size[:, -self.rope:] * 2.0 ** -18 + np.abs(y[:, -self.rope:]) * 2.0 ** -8 * 1.01 + 1e-37).all()
            n += length
        return n


STEPS = [[60, 0, 23], [1, 31, 1], "evict", [1, 1, 1], [1, 20, 1], "evict", [1, 1, -1], [1, 1, 40], "evict", [1, 1, 1]]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("nope,rope", [(512, 64), (256, 0)])
def test_rotation_after_evictions(gpu, nope, rope, kind):
    s = Sequences(gpu, kind, nope, rope)
    rows = 0
    for step in STEPS:
        if step == "evict":
            s.evict(17)
        else:
            s.grow(step)
        rows += s.check_rows()
    assert rows > 300 and s.err.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF16, FP8])
def test_distance_bias_after_evictions(gpu, kind):
    """The attention's bias by the distance of the tokens' places, over what two evictions left."""
    s = Sequences(gpu, kind, 256, 0)
    slopes = torch.tensor([2.0 ** -(i / 2) for i in range(16)], device=gpu)
    for step in STEPS:
        if step == "evict":
            s.evict(17)
            continue
        x, _, req, pos, tlen, place = s.grow(step)
        out = dsa.dsa_paged_attn(x, s.cache, kind, s.table, tlen, 1 / 16, page_size=s.page, req_of_token=req, slopes=slopes,
                                 q_positions=place, key_positions=s.kpos, error_word=s.err)
        torch.cuda.synchronize()
        c = s.cache.cpu()
        rows = c.numpy() if kind == FP8 else c.view(torch.int16).numpy().view(np.uint16)
        table = s.table.cpu().numpy()
        for t in range((tlen > 0).sum().item()):
            r, n = req[t].item(), tlen[t].item()
            kp = s.kpos.cpu().numpy()
            u, k, _, _ = G.scores(x[t].cpu().double().numpy(), rows, table, s.page, r, 0, n, 1 / 16, 0.0, slopes.cpu().numpy(),
                                  len(s.keys[r]) - (tlen[req == r].max().item() - n) - 1, kp)
            o, _, pk, spread = G.softmax_output(u, k)
            tol = np.abs(o) * 2.0 ** -8 + 2.0 ** -8 * spread * 2 + pk * 2.0 ** -9
            assert (np.abs(out[t].cpu().double().numpy() - o) <= tol + 1e-6).all(), t
    assert s.err.item() == 0
