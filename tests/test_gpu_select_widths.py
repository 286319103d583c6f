"""The choice of blocks at the widths where its variant changes, each full and one past it, and calls that it
refuses."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from oracle import steps as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [16385, (1 << 31) - 1])
def test_no_room_is_made_for_a_refused_choice(gpu, K):
    scores, table = torch.zeros((64, 4), device=gpu), torch.zeros((64, 4), dtype=torch.int32, device=gpu)
    lens = torch.zeros(64, dtype=torch.int32, device=gpu)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(dsa.DsaError):
        dsa.dsa_block_select(scores, table, lens, K, page_size=16)
    assert torch.cuda.max_memory_allocated() == before


# the blocks that each variant holds, and one past the largest
LIMITS = [160, 288, 544, 1152, 2304, 4608, 8704]


@pytest.mark.parametrize("K", ["few", "half", "all but one", "all", "more"])
@pytest.mark.parametrize("width", [w + d for w in LIMITS for d in (-1, 0, 1)])
def test_capacity(gpu, width, K):
    rng = np.random.default_rng(width)
    K = {"few": 7, "half": width // 2, "all but one": width - 1, "all": width, "more": width + 3}[K]
    sink, recent = (1, 2) if K < 10 else (0, 0)
    page, T = 4, 6
    # full rows (the last block full, and of one position), the last register's and word's neighbours, a short and an empty one
    lens = [width * page, width * page - 3, (width - 1) * page, (width - 33) * page, 50, 0]
    table = rng.permutation(2 * width).astype(np.int32).reshape(2, width)
    req = [0, 1, 1, 0, 1, 0]
    s = np.exp(rng.standard_normal((T, width))).astype(np.float32)
    s[rng.random(s.shape) < 0.2] = 1.5
    s[rng.random(s.shape) < 0.05] = -0.0
    s[rng.random(s.shape) < 0.05] = 0.0
    s[1, -1] = 100.0  # the last key is the best
    s[2, width - 2] = -100.0  # and the worst
    for t, n in enumerate(lens):
        s[t, -(-n // page):] = np.nan
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=gpu)  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    got = dsa.dsa_block_select(torch.from_numpy(s).to(gpu), i32(table), i32(lens), K, page_size=page, req_of_token=i32(req),
                               sink=sink, recent=recent, error_word=err)
    blocks, own, out = (x.cpu().numpy() for x in got)
    assert err.item() == 0
    for t, n in enumerate(lens):
        want = S.select(s[t], -(-n // page), K, sink, recent)
        m = len(want)
        assert blocks[t, :m].tolist() == want and (blocks[t, m:] == -1).all(), t
        assert own[t, :m].tolist() == table[req[t], want].tolist() and (own[t, m:] == -1).all(), t
        assert out[t] == sum(min(page, n - b * page) for b in want), t


@pytest.mark.parametrize("width", LIMITS)
def test_equal_scores_at_capacity(gpu, width):
    """All keys equal: the first K blocks, up to the last key of a full row."""
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=gpu)  # noqa: E731
    for w in (width, width + 1):
        for K in (1, w - 1, w):
            blocks, own, out = dsa.dsa_block_select(torch.zeros((1, w), device=gpu), i32(np.arange(w)[None] + 5), i32([w]), K,
                                                    page_size=1, recent=0)
            assert torch.equal(blocks[0].cpu(), torch.arange(K, dtype=torch.int32)) and torch.equal(own, blocks + 5)
            assert out.item() == K
