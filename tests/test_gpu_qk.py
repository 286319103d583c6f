"""Norms, rotation and the cache write on the GPU against fp64 (oracle/steps.py).

Tolerances, from the roundings. fp32: the sum of squares adds at most 18 terms in a chain and five
levels over the lanes (23 * 2^-24 of it, half of that in the root), its mean, the reciprocal root (2
ulp) and two products: below 2^-19 of the value. The angles' products add 2^-23 of |a| + |b|. So a
column errs by less than e32 = 2^-18 * size, size = |y|, or |a| + |b| where it was turned; rounding
to bf16 adds half a step, 2^-8 |y|. A packed column errs by e32, half an e4m3 step (2^-4 |y|, or 2^-10 of
the tile's scale below the smallest normal code) and what the division adds (2^-23); the scale by 2^-18."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from oracle import paged as G
from oracle import steps as S

pytestmark = pytest.mark.gpu

BF16, FP8 = dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED
EPS = 1e-6


def f64(t):
    return t.detach().cpu().double().numpy()


def angles_table(gen, n, dev):
    a = torch.rand((n, 32), generator=gen, device=dev) * 6.3
    return torch.cat([a.cos(), a.sin()], dim=1)


def near(got, y, size, what, step=2.0 ** -8, floor=0.0):
    assert got.shape == y.shape
    if y.size == 0:
        return
    tol = size * 2.0 ** -18 + np.abs(y) * step * (1 + 2.0 ** -7) + floor + 1e-37
    off = np.abs(got - y) - tol
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off[at] <= 0, (what, at, got[at], y[at], tol[at])


def near_cache(cache, kind, nope, slots, y, size, what):
    rows = cache[slots]
    if len(slots) == 0:
        return
    if kind == BF16:
        near(f64(rows), y, size, what)
        return
    raw = rows.cpu().numpy()
    tiles = nope // 128
    scale = np.ascontiguousarray(raw[:, nope:nope + 4 * tiles]).view(np.float32).astype(np.float64)
    amax = np.abs(y[:, :nope]).reshape(-1, tiles, 128).max(axis=2)
    room = size[:, :nope].reshape(-1, tiles, 128).max(axis=2)
    assert (np.abs(scale - amax / 448) <= room / 448 * 2.0 ** -18).all(), what
    wide = np.repeat(scale, 128, axis=1)
    near(G.E4M3[raw[:, :nope]] * wide, y[:, :nope], size[:, :nope], what, 2.0 ** -4, wide * 2.0 ** -10 * 1.01)
    if y.shape[1] > nope:
        tail = np.ascontiguousarray(raw[:, nope + 4 * tiles:]).view(np.uint16)
        near(G.P.bf16_to_f64(tail), y[:, nope:], size[:, nope:], what)


def check(dev, T, H, kind=FP8, rope=64, q_norm=None, k_norm=None, rotate=True, inter=False, weights=True, pad=(),
          inplace=False, strided=False, seed=0, eps=EPS, scale=1.0, no_loc=False):
    gen = torch.Generator(device=dev).manual_seed(seed)
    nope = 512 if rope else 256
    D = nope + rope
    row = D if kind == BF16 else nope + nope // 32 + 2 * rope
    slots = T + 9
    bf = dict(dtype=torch.bfloat16, device=dev)

    def tensor(*shape):
        if not strided:
            return torch.randn(shape, generator=gen, device=dev).mul(scale).to(torch.bfloat16)
        big = torch.full((*shape[:-1], shape[-1] + 24), float("nan"), **bf)
        v = big[..., 8:8 + shape[-1]]
        v.copy_(torch.randn(shape, generator=gen, device=dev) * scale)
        return v

    q, k = (tensor(T, H, D) if H else None), tensor(T, D)
    pos = torch.randint(0, 300, (T,), generator=gen, device=dev).to(torch.int32)
    if T:
        pos[0] = 299
    for i in pad:
        pos[i] = -1 - i
    cs = angles_table(gen, 300, dev) if rope and rotate else None
    loc = torch.randperm(slots, generator=gen, device=dev)[:T]
    qn = D if q_norm is None else q_norm
    kn = nope if k_norm is None else k_norm
    qw = (1 + 0.2 * torch.randn(qn, generator=gen, device=dev)).to(torch.bfloat16) if weights and qn else None
    kw = (1 + 0.2 * torch.randn(kn, generator=gen, device=dev)).to(torch.bfloat16) if weights and kn else None
    cache = torch.full((slots, row), 7, dtype=torch.uint8 if kind == FP8 else torch.bfloat16, device=dev)
    before = cache.clone()
    xq, xk = (f64(q) if H else None), f64(k)
    out = None
    if H:
        out = q if inplace else torch.full((T, H, D), 5.0, **bf)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = dsa.dsa_qk_norm_rope(q, k, pos, cs, eps, cache, kind, None if no_loc else loc, d_nope=nope, d_rope=rope, q_norm=qn,
                               k_norm=kn, q_weight=qw, k_weight=kw, interleaved=inter, q_out=out, error_word=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and got is out
    live = pos.cpu().numpy() >= 0
    ang = None if cs is None else f64(cs)[np.maximum(pos.cpu().numpy(), 0)]
    if H:
        y, size = S.norm_rope(xq, qn, None if qw is None else f64(qw), eps, None if ang is None else ang[:, None], inter)
        near(f64(got)[live], y[live], size[live], "q")
        rest = xq if inplace else np.full_like(xq, 5.0)
        assert np.array_equal(f64(got)[~live], rest[~live])
    y, size = S.norm_rope(xk, kn, None if kw is None else f64(kw), eps, ang, inter)
    at = np.arange(T) if no_loc else loc.cpu().numpy()
    near_cache(cache, kind, nope, torch.from_numpy(at[live]).to(dev), y[live], size[live], "k")
    others = np.setdiff1d(np.arange(slots), at[live])
    assert torch.equal(cache[others], before[others])


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("rope,inter", [(0, False), (64, False), (64, True)])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (3, 5), (70, 64)])
def test_shapes(gpu, T, H, rope, inter, kind):
    check(gpu, T, H, kind, rope, inter=inter, seed=T + H)


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("which", range(3))
def test_what_the_norm_covers(gpu, rope, weights, which):
    nope = 512 if rope else 256
    n = [0, nope, nope + rope]
    for kind in (BF16, FP8):
        check(gpu, 9, 6, kind, rope, q_norm=n[which], k_norm=n[(which + 1) % 3], weights=weights, rotate=which != 1)


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("rope", [0, 64])
def test_in_place_strided_padded(gpu, kind, rope):
    check(gpu, 12, 3, kind, rope, inplace=True, pad=(0, 5, 11))
    check(gpu, 12, 3, kind, rope, strided=True, pad=(1,))
    check(gpu, 12, 3, kind, rope, strided=True, inplace=True)
    check(gpu, 5, 0, kind, rope, no_loc=True)
    check(gpu, 0, 4, kind, rope)


@pytest.mark.parametrize("scale", [1e-18, 1e-3, 1e4, 1e17])
def test_magnitudes(gpu, scale):
    for kind in (BF16, FP8):
        check(gpu, 6, 4, kind, scale=scale, eps=1e-30 if scale < 1 else 1e-6)
        check(gpu, 6, 4, kind, scale=scale, eps=1e3)


def test_heads_by_tokens_layout(gpu):
    """Queries as [H, T, D] in memory, the result too."""
    gen = torch.Generator(device=gpu).manual_seed(3)
    q = torch.randn((8, 5, 256), generator=gen, device=gpu).to(torch.bfloat16).transpose(0, 1)
    out = torch.empty((8, 5, 256), dtype=torch.bfloat16, device=gpu).transpose(0, 1)
    got = dsa.dsa_qk_norm_rope(q, q_norm=256, q_out=out)
    y, size = S.norm_rope(f64(q), 256, None, 1e-6, None, False)
    near(f64(got), y, size, "q")


def test_zero_rows_and_a_single_peak(gpu):
    k = torch.zeros((3, 576), dtype=torch.bfloat16, device=gpu)
    k[1, 200] = 3.0
    k[2, :512] = -0.0
    cache = torch.full((3, 656), 9, dtype=torch.uint8, device=gpu)
    dsa.dsa_qk_norm_rope(k=k, cache=cache, kind=FP8, d_nope=512, d_rope=64, k_norm=512)
    want = dsa.dsa_quant_k_cache(torch.zeros((1, 512), dtype=torch.bfloat16, device=gpu),
                                 torch.zeros((1, 64), dtype=torch.bfloat16, device=gpu))
    assert torch.equal(cache[0], want[0])
    assert (cache[2, 512:528] == 0).all()
    scale = cache[1, 512:528].view(torch.float32)
    assert scale[0] == scale[2] == scale[3] == 0 and abs(scale[1].item() * 448 - 512 ** 0.5) < 1e-4 * 512 ** 0.5
    assert cache[1, 200].item() == 0x7E and (cache[1, :128] == 0).all()


def test_without_a_norm_the_row_is_packed_as_the_pack_packs(gpu):
    gen = torch.Generator(device=gpu).manual_seed(5)
    for nope, rope in ((256, 0), (512, 64)):
        k = (torch.randn((50, nope + rope), generator=gen, device=gpu) * 3).to(torch.bfloat16)
        loc = torch.randperm(60, generator=gen, device=gpu)[:50]
        want = dsa.dsa_quant_k_cache(k[:, :nope], k[:, nope:] if rope else None, out_loc=loc, num_slots=60)
        got = torch.zeros_like(want)
        dsa.dsa_qk_norm_rope(k=k, cache=got, kind=FP8, out_loc=loc, d_nope=nope, d_rope=rope)
        assert torch.equal(got, want)


def test_bad_positions_and_slots(gpu):
    gen = torch.Generator(device=gpu).manual_seed(6)
    q = torch.randn((5, 4, 576), generator=gen, device=gpu).to(torch.bfloat16)
    k = torch.randn((5, 576), generator=gen, device=gpu).to(torch.bfloat16)
    cs = angles_table(gen, 10, gpu)
    pos = torch.tensor([0, 10, 2, -1, 9], dtype=torch.int32, device=gpu)
    loc = torch.tensor([0, 1, -5, 3, 8], device=gpu)
    args = dict(d_nope=512, d_rope=64, q_norm=576, k_norm=512)

    def run(pos, loc):
        out, cache = torch.full_like(q, 2.0), torch.full((8, 576), 2.0, dtype=torch.bfloat16, device=gpu)
        err = torch.zeros(1, dtype=torch.int32, device=gpu)
        dsa.dsa_qk_norm_rope(q, k, pos, cs, 1e-6, cache, BF16, loc, q_out=out, error_word=err, **args)
        return (out != 2.0).flatten(1).any(1).tolist(), (cache != 2.0).any(1).nonzero().flatten().tolist(), err.item()

    assert run(pos, loc) == ([True, False, True, False, True], [0],
                             dsa.DEVERR_INDEX_OUT_OF_RANGE | dsa.DEVERR_SLOT_OUT_OF_RANGE)
    assert run(pos.clamp(max=9), loc.clamp(max=7)) == ([True, True, True, False, True], [0, 1, 7], 0)
    # the error word is optional
    dsa.dsa_qk_norm_rope(q, k, pos, cs, 1e-6, torch.zeros((8, 576), dtype=torch.bfloat16, device=gpu), BF16, loc, **args)
    torch.cuda.synchronize()


def test_slots_past_four_gigabytes(gpu):
    slots = (1 << 32) // 264 + 1000
    cache = torch.zeros((slots, 264), dtype=torch.uint8, device=gpu)
    k = torch.randn((4, 256), device=gpu).to(torch.bfloat16)
    loc = torch.tensor([slots - 1, 0, slots - 500, 5], device=gpu)
    dsa.dsa_qk_norm_rope(k=k, cache=cache, kind=FP8, out_loc=loc, k_norm=256)
    small = torch.zeros((4, 264), dtype=torch.uint8, device=gpu)
    dsa.dsa_qk_norm_rope(k=k, cache=small, kind=FP8, k_norm=256)
    assert torch.equal(cache[loc], small)


def test_repeats_streams_and_graphs(gpu):
    gen = torch.Generator(device=gpu).manual_seed(8)
    q = torch.randn((33, 7, 576), generator=gen, device=gpu).to(torch.bfloat16)
    k = torch.randn((33, 576), generator=gen, device=gpu).to(torch.bfloat16)
    cs, pos = angles_table(gen, 50, gpu), torch.arange(33, dtype=torch.int32, device=gpu)
    args = dict(d_nope=512, d_rope=64, q_norm=512, k_norm=576)

    def run(cache):
        return dsa.dsa_qk_norm_rope(q, k, pos, cs, 1e-6, cache, FP8, **args)

    caches = [torch.zeros((40, 656), dtype=torch.uint8, device=gpu) for _ in range(3)]
    first = run(caches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run(caches[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = run(caches[2])
    pos.copy_(pos + 3)
    want_cache = torch.zeros_like(caches[2])
    want = run(want_cache)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(caches[0], caches[1])
    assert torch.equal(third, want) and torch.equal(caches[2], want_cache)


def test_binding_refusals(gpu):
    q = torch.zeros((2, 3, 576), dtype=torch.bfloat16, device=gpu)
    k, w = q[:, 0], torch.ones(576, dtype=torch.bfloat16, device=gpu)
    cache = torch.zeros((4, 656), dtype=torch.uint8, device=gpu)
    pos, cs = torch.zeros(2, dtype=torch.int32, device=gpu), torch.zeros((5, 64), device=gpu)
    geo = dict(d_nope=512, d_rope=64)
    for kw in (dict(q=q), dict(q=q.float(), **geo), dict(q=q, q_norm=576, q_weight=w[:512], **geo), dict(k=k, **geo),
               dict(k=k, cache=cache, kind=BF16, **geo), dict(k=k[:1], q=q, cache=cache, kind=FP8, **geo),
               dict(q=q, q_out=q[:, :2], **geo), dict(q=q, positions=pos[:1], **geo),
               dict(q=q, positions=pos, cos_sin=cs[:, :32], **geo), dict(k=k, cache=cache, kind=FP8, q_out=q, **geo),
               dict(q=q.transpose(1, 2), **geo), dict(q=q, positions=pos.cpu(), **geo), dict(q=q, q_norm=1 << 32, **geo)):
        with pytest.raises(ValueError):
            dsa.dsa_qk_norm_rope(**kw)
    for kw in (dict(q=q, cos_sin=cs, **geo), dict(q=q, q_norm=100, **geo), dict(q=q, eps=0.0, **geo)):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_qk_norm_rope(**kw)
