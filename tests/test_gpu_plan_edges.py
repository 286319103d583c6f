"""The batch plan where pages have several holders."""
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa

pytestmark = pytest.mark.gpu


def test_requests_that_share_their_first_pages(gpu):
    """Ended as the header says, a shared page goes back once, with its last holder; ended at once, twice."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    page, shared = 16, 2

    def state():
        return dict(lengths=i32([2 * page + 5, 2 * page + 20, 0]), held=i32([3, 4, 0]),
                    block_table=i32([[7, 4, 1, -1], [7, 4, 9, 2], [-1] * 4]), free_pages=i32([3, 5] + [-1] * 8),
                    num_free=i32([2]))

    def step(s, new):
        dsa.dsa_batch_plan(s["lengths"], i32(new), s["held"], s["block_table"], s["free_pages"], s["num_free"], 64,
                           page_size=page)
        return s["free_pages"][:s["num_free"].item()].tolist()

    s = state()
    s["lengths"][0] = shared * page
    assert step(s, [0, 1, 0]) == [3, 5, 1]  # the other goes on
    s["lengths"][0] = s["held"][0] = 0
    assert s["block_table"][1].tolist() == [7, 4, 9, 2] and s["lengths"].tolist() == [0, 2 * page + 21, 0]
    assert step(s, [0, 0, 20]) == [3] and s["block_table"][2, :2].tolist() == [1, 5]
    assert step(s, [0, -1, 0]) == [3, 7, 4, 9, 2]  # the last holder
    s = state()
    assert step(s, [-1, -1, 0]) == [3, 5, 7, 4, 1, 7, 4, 9, 2]


@pytest.mark.parametrize("tokens", [(1 << 30) + 1, (1 << 31) - 1, (1 << 40), -1])
def test_no_room_is_made_for_a_refused_number_of_tokens(gpu, tokens):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    args = (i32([1]), i32([1]), i32([1]), i32([[0, 1]]), i32([2]), i32([1]))
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(ValueError):
        dsa.dsa_batch_plan(*args, tokens, page_size=16)
    assert torch.cuda.max_memory_allocated() == before
