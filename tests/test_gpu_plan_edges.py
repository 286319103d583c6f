"""The batch plan where pages have several holders, where requests are refused in a cluster or over several
passes of requests, and at the borders of its launches."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from test_gpu_plan import check, pages

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


def refused_steps(R, page, most, ends, first_pages, first_tokens, seed):
    """(lengths, new tokens, held, free pages, room): pages run out at request `first_pages` or a little behind it,
    room at `first_tokens`."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 60, R)
    held = np.array([pages(int(n), page) for n in lens])
    new = rng.integers(1, most + 1, R)
    new[5:5 + ends] = -1
    lens[20:40] //= 2  # these were evicted, and give pages back
    add = np.maximum(new, 0)
    need = np.array([pages(int(n + m), page) for n, m in zip(lens, add)])
    need[new < 0] = 0
    take, back = np.maximum(need - held, 0), np.maximum(held - need, 0)
    first_pages += int(np.argmax(take[first_pages:] > 0))  # it wants some
    spare = int(take[:first_pages].sum() - back.sum())
    room = int(add[:first_tokens].sum())
    assert spare >= 0 and take[first_pages] > 0
    return lens.tolist(), new.tolist(), held.tolist(), spare, room


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("R,most,first_pages,first_tokens", [
    (2500, 12, 1500, 2200),   # pages run out in the second pass over the requests, room in the third
    (2500, 12, 2100, 300),    # room in the first, pages (which refused requests want too) in the last
    (1025, 30, 1023, 1024),   # at the border of a pass
    (1024, 30, 600, 900),     # the cluster, full
    (300, 12, 120, 200), (300, 12, 250, 90), (300, 99, 100, 290)])
def test_refusals_where_sums_are_carried(gpu, R, most, first_pages, first_tokens, inplace):
    page = 8
    lens, new, held, spare, room = refused_steps(R, page, most, 9, first_pages, first_tokens, R + most)
    check(gpu, lens, new, held, room, page, width=40, spare=spare, inplace=inplace,
          want_err=dsa.DEVERR_OUT_OF_PAGES | dsa.DEVERR_TOKEN_CAPACITY)


@pytest.mark.parametrize("T", [1024, 1025, 16383, 16384, 16385])
@pytest.mark.parametrize("R", [3, 700, 1500])
def test_borders_of_the_launches(gpu, R, T):
    """Room for as many tokens as the plan's own blocks write, one less and one more, full and nearly."""
    new = [T // R] * R
    new[-1] += T - sum(new)
    for less in (0, 1):
        new[0] -= less
        check(gpu, [5] * R, new, [1] * R, T, 16, width=max(new) // 16 + 3, spare=sum(n // 16 + 2 for n in new))
    new[0] += 2
    check(gpu, [5] * R, new, [1] * R, T, 16, width=max(new) // 16 + 3, spare=sum(n // 16 + 2 for n in new),
          want_err=dsa.DEVERR_TOKEN_CAPACITY)
