"""Dense paged attention and its mass where a score, a scale or a component is far from the others,
against the fp64 definitions (oracle/paged.py).

Tolerances, per element (u = 2^-24 fp32, 2^-8 bf16 half steps):
  score    d = 256 * 2^-23 * B + 2^-19 |u|, B = max_j |sm_scale| sum |q k| (an fp32 sum of 256 exact
           products in any order, one step of slack for truncation; then cap, bias and the change to
           base 2: below 2^-19 of the score's parts, the exponential of the cap's long branch
           amplified by 1 / sinh(2 |u| / cap) < 2); with an FP8 cache
           + 2^-17 |sm_scale| max |q| max_j sum |k| over the columns in which q is not zero (half of the
           query's smallest second step)
  lse, out, mass: as in test_gpu_paged.py, from this d
"""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from oracle import paged as R
from oracle import projection as P

from _helpers import f32_of
from test_gpu_paged import Case, dev_t

pytestmark = pytest.mark.gpu

BF16, FP8 = dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED


def score_error(c, t, u, k, bias):
    """[H] bound of the scores' error."""
    if u.shape[1] == 0:
        return np.zeros(c.H)
    q = P.bf16_to_f64(c.q[t])
    d = 256 * 2.0 ** -23 * (np.abs(q) @ np.abs(k).T).max(axis=1) * abs(c.sm_scale)
    d = d + 2.0 ** -19 * (np.abs(u).max(axis=1) + bias)
    if c.kind == FP8:
        d = d + 2.0 ** -17 * abs(c.sm_scale) * np.abs(q).max(axis=1) * ((q != 0) @ np.abs(k).T).max(axis=1)
    return d


def run_and_check(c, cap=0.0, slopes=None, qpos=None, mass=True):
    dev, T = c.dev, len(c.lens)
    opts = c.opts(logit_cap=cap, slopes=dev_t(slopes, dev), q_positions=dev_t(qpos, dev))
    lse = torch.full((T, c.H), float("nan"), device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = dsa.dsa_paged_attn(*c.args(), lse=lse, error_word=err, **opts)
    m0 = np.random.default_rng(5).random((T, int(c.lens.max()) + 3)).astype(np.float32)
    weights = torch.from_numpy(m0).to(dev)
    if mass:
        dsa.dsa_paged_attn_mass(*c.args(), lse, weights, error_word=err, **opts)
    torch.cuda.synchronize()
    assert err.item() == 0
    got, gl = f32_of(out).astype(np.float64), lse.cpu().numpy().astype(np.float64)
    got_m = weights.cpu().numpy().astype(np.float64)
    for t in range(T):
        b = int(c.lens[t])
        qp = b - 1 if qpos is None else int(qpos[t])
        u, k, pos, _ = R.scores(P.bf16_to_f64(c.q[t]), c.cache, c.bt, c.page, t, 0, b, c.sm_scale,
                                float(np.float32(cap)), slopes, qp)
        n = len(pos)
        bias = 0.0 if slopes is None else np.abs(slopes).max() * np.abs(qp - pos).max()
        d = score_error(c, t, u, k, bias)
        ref, rl, absum, l2 = R.softmax_output(u, k)
        e = np.abs(gl[t] - rl)
        assert (e <= d + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl)).all(), (t, e.max(), d.max())
        tol = 2.0 ** -8 * np.abs(ref) + 5 * 2.0 ** -8 * l2 + (2 * d[:, None] + n * 2.0 ** -22 + 2.0 ** -20) * absum
        e = np.abs(got[t] - ref)
        assert (e <= tol).all(), (t, np.unravel_index(np.argmax(e - tol), e.shape), (e / np.maximum(tol, 1e-300)).max())
        if mass:
            w = np.exp(u - gl[t][:, None])
            tol = (w * (d[:, None] + 2.0 ** -20)).sum(axis=0) + (c.H + 2) * 2.0 ** -24 * np.abs(m0[t, pos] + w.sum(axis=0))
            e = np.abs(got_m[t, pos] - (m0[t, pos] + w.sum(axis=0)))
            assert (e <= tol).all(), (t, (e / tol).max())
    return out, lse


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("cap", [1e-40, 1e-3, 2.0, 1e3, 1e6, 1e9, 1e30, 3e38])
def test_caps_of_every_size(gpu, kind, cap):
    """A cap far above the scores leaves them as they are, whatever its size; one far below them
    makes them all equal in magnitude. Scores of exactly zero among them."""
    c = Case(gpu, kind, [1, 700], 16, seed=83)
    c.q[:, 3] = 0
    run_and_check(c, cap=cap)


def _far_scales(dev, n, at, exponent, both, H=16):
    """n FP8 keys whose first tile has scale 2^-exponent, except the key at position `at`: scale 1 and a
    score near -60 (odd heads, if `both`: 60). Scores come from the second tile alone."""
    c = Case(dev, FP8, [n], H, seed=exponent + at)
    rng = np.random.default_rng(at)
    c.cache[:, :256] &= 0x7F
    c.cache[:, :256] = np.minimum(c.cache[:, :256], 0x7E) | (rng.integers(0, 2, (len(c.cache), 256)) << 7).astype(np.uint8)
    scale = np.tile(np.array([2.0 ** -exponent, 1.0 / 448], dtype=np.float32), (len(c.cache), 1))
    q = np.zeros((1, H, 256))
    q[:, :, 128:] = rng.choice([-1.0, 1.0], 128) + 0.1 * rng.standard_normal((1, H, 128))
    if both:
        q[:, 1::2] *= -1
    c.q = P.f64_to_bf16(q)
    c.sm_scale = 0.5
    slot = R.slots_of(c.bt, c.page, len(c.cache), 0, np.arange(n))
    scale[slot[at], 0] = 1.0
    # all of the key's second tile against the query's signs: 0.5 * 128 * 0.9375 = 60
    scale[slot[at], 1] = 1.0
    one = np.where(q[0, 0, 128:] > 0, 0xB7, 0x37).astype(np.uint8)  # -+0.9375
    c.cache[slot[at], 128:256] = one
    c.cache[:, 256:] = scale.view(np.uint8).reshape(-1, 8)
    return c


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("exponent", [8, 20, 24, 28, 33, 40])
@pytest.mark.parametrize("n,at", [(400, 5), (400, 399), (3000, 1500)])
def test_a_large_scale_of_no_weight(gpu, n, at, exponent, both):
    """The output keeps its precision beside a key of large scale that the softmax ignores, before and
    behind the others, and whether or not other heads attend to that key."""
    run_and_check(_far_scales(gpu, n, at, exponent, both))


def test_scales_that_grow_along_the_range(gpu):
    """Scales rise and fall by 2^60 over the range, in both tiles, under a flat and a sharp softmax."""
    for sm in (1e-4, 1.0):
        c = Case(gpu, FP8, [50, 3000], 16, seed=89)
        for r in range(2):
            slot = R.slots_of(c.bt, c.page, len(c.cache), r, np.arange(c.lens[r]))
            x = np.abs(np.linspace(-1, 1, len(slot)))
            c.cache[slot, 256:] = np.exp2(-60 * np.stack([x, 1 - x], axis=1)).astype(np.float32).view(np.uint8).reshape(-1, 8)
        c.sm_scale = sm
        run_and_check(c)


@pytest.mark.parametrize("exponent", [-100, -60, 100])
def test_scales_of_every_size(gpu, exponent):
    """All scales far from 1, where references meet their limits, and a first tile without any."""
    c = Case(gpu, FP8, [50, 1500], 16, seed=103)
    scale = np.exp2(exponent + np.random.default_rng(3).uniform(-1, 1, (len(c.cache), 2))).astype(np.float32)
    slot = R.slots_of(c.bt, c.page, len(c.cache), 1, np.arange(256))
    scale[slot] = 0.0
    if exponent == -100:  # (below 2^-80 precision may fall: what is left has to be finite and small)
        c.cache[:, 256:] = scale.view(np.uint8).reshape(-1, 8)
        out = dsa.dsa_paged_attn(*c.args(), **c.opts())
        assert (f32_of(out)[1] == 0).sum() < out[1].numel() and np.abs(f32_of(out)).max() < 2.0 ** -90
        return
    c.cache[:, 256:] = scale.view(np.uint8).reshape(-1, 8)
    c.sm_scale = 2.0 ** -exponent / 4000
    run_and_check(c)


@pytest.mark.parametrize("H", [1, 64])
def test_query_components_far_below_the_largest(gpu, H):
    """Components below 2^-9 of the head's largest err by at most 2^-17 of it: keys that read these
    components alone add up their errors. Half the heads hold the component that a split of both terms
    at the same step errs by 1.94 times as much on."""
    c = Case(gpu, FP8, [1, 1, 130], H, seed=97)
    c.cache[:, :256] = 0x38
    c.cache[:, 0] = 0
    c.cache[:, 256:] = np.ones((len(c.cache), 2), dtype=np.float32).view(np.uint8)
    q = np.full((3, H, 256), 0.00970458984375 / 128)
    q[:, 1::2] = np.exp(np.random.default_rng(1).uniform(-14, -5, q[:, 1::2].shape))
    q[:, :, 0] = 1.0
    c.q = P.f64_to_bf16(q)
    c.sm_scale = 1.0
    run_and_check(c)


@pytest.mark.parametrize("kind", [BF16, FP8])
@pytest.mark.parametrize("lens", [[1, 7], [130, 5000]])
def test_scores_far_below_zero(gpu, kind, lens):
    """All scores of a head below -1e30: the largest still takes all of the weight, in one part or
    joined from many."""
    c = Case(gpu, kind, lens, 3, seed=101)
    slopes = np.array([2e31, 0.0, 3e33], dtype=np.float32)
    out, lse = run_and_check(c, slopes=slopes, qpos=np.array([9000, 9001], dtype=np.int32), mass=False)
    for t, n in enumerate(lens):
        k = R.latent_rows(c.cache, R.slots_of(c.bt, c.page, len(c.cache), t, [n - 1]))[0]
        assert (np.abs(f32_of(out)[t, [0, 2]] - k) <= 2.0 ** -8 * np.abs(k)).all()
