"""Packed key rows of dsa_qk_norm_rope at the ends of the number range."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa

pytestmark = pytest.mark.gpu

FP8 = dsa.CACHE_FP8_SCALED


def packed(k, nope, rope, **kw):
    """(packed rows, the rows as bf16) of k [T, nope + rope]."""
    cache = torch.full((k.shape[0], nope + nope // 32 + 2 * rope), 9, dtype=torch.uint8, device=k.device)
    dsa.dsa_qk_norm_rope(k=k, cache=cache, kind=FP8, d_nope=nope, d_rope=rope, **kw)
    at = torch.arange(k.shape[0], dtype=torch.int32, device=k.device)
    return cache, dsa.dsa_gather_dequant(cache, FP8, nope, rope, at)


@pytest.mark.parametrize("nope,rope", [(256, 0), (512, 64)])
@pytest.mark.parametrize("whole", [False, True])
def test_nan_stays_nan(gpu, nope, rope, whole):
    """A NaN under the norm makes every normalised column NaN, an infinity its own (the others are x * 0): as
    codes too, whose tiles have no largest value then."""
    n = nope + rope if whole else nope
    k = torch.ones((5, nope + rope), dtype=torch.bfloat16, device=gpu)
    k[1, 3] = float("nan")
    k[2, nope - 1] = float("inf")
    k[3, 130] = -float("inf")
    if rope:
        k[4, nope + 5] = float("nan")
    cache, rows = packed(k, nope, rope, k_norm=n)
    bad = rows.isnan().cpu().numpy()
    want = np.zeros((5, nope + rope), dtype=bool)
    want[1, :n] = True
    want[2, nope - 1] = want[3, 130] = True
    if rope:
        want[4, nope + 5] = True
        if whole:
            want[4] = True
    assert np.array_equal(bad, want)
    got = rows.float().cpu().numpy()
    assert (np.abs(got[0] - 1) < 2.0 ** -4).all()
    assert (got[2:4, :nope][~want[2:4, :nope]] == 0).all()
    # bf16 rows say the same
    plain = torch.zeros((5, nope + rope), dtype=torch.bfloat16, device=gpu)
    dsa.dsa_qk_norm_rope(k=k, cache=plain, kind=dsa.CACHE_BF16, d_nope=nope, d_rope=rope, k_norm=n)
    assert np.array_equal(plain.isnan().cpu().numpy(), want)


def test_nan_without_a_norm(gpu):
    """Beside finite columns as the pack does it; a tile of nothing else keeps its NaN."""
    k = torch.ones((3, 256), dtype=torch.bfloat16, device=gpu)
    k[0, 7] = float("nan")
    k[1, :128] = float("nan")
    k[2, :128] = 0.0
    k[2, 9] = float("nan")
    cache, rows = packed(k, 256, 0)
    assert torch.equal(cache[0], dsa.dsa_quant_k_cache(k)[0])
    assert rows.isnan().sum(1).tolist() == [1, 128, 1]
    assert rows[0, 7].isnan() and rows[1, :128].isnan().all() and rows[2, 9].isnan() and (rows[2, 10:128] == 0).all()


@pytest.mark.parametrize("value", [2.0 ** -10, 2.0 ** -7, 1.0, 200.0])
def test_rows_below_the_smallest_scale_are_zero(gpu, value):
    """The smallest bf16 weight makes products of a few units of the last place of fp32, whose 448th part can round
    to no scale at all: the row is finite then, and off by less than 448 halves of the smallest fp32 number."""
    k = torch.zeros((2, 256), dtype=torch.bfloat16, device=gpu)
    k[0, 5], k[0, 9], k[1, 200] = value, -value / 2, value
    w = torch.full((256,), 2.0 ** -133, dtype=torch.bfloat16, device=gpu)
    cache, rows = packed(k, 256, 0, k_norm=256, k_weight=w, eps=1.0)
    x = k.double()
    want = x * (x.square().mean(1, keepdim=True) + 1).rsqrt() * 2.0 ** -133
    codes = cache[:, :256].view(torch.float8_e4m3fn).float().double()
    scales = cache[:, 256:].contiguous().view(torch.float32).double().repeat_interleave(128, dim=1)
    assert codes.isfinite().all() and rows.isfinite().all()
    # half a step of a scale of 2^-149 steps times a code, half a code's step, and the fp32 product's own half step
    off = (codes * scales - want).abs()
    assert (off <= 448 * 2.0 ** -150 + want.abs() * 2.0 ** -4 + 2.0 ** -149).all()
