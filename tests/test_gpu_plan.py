"""The batch plan on the GPU against its definition (oracle/steps.py): every output, every table entry
and the free stack equal, with each kind of refusal, in place and not, from a captured graph."""
import numpy as np
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from oracle import steps as S

pytestmark = pytest.mark.gpu

BAD = dsa.DEVERR_INDEX_OUT_OF_RANGE
NAMES = ("cu", "req", "positions", "token_lengths", "out_loc")


def build(rng, lens, held, width, spare, room=None):
    """(table, stack, entries on it): the requests' pages and the free ones, all different."""
    R = len(lens)
    n = [min(max(h, 0), width) for h in held]
    perm = rng.permutation(sum(n) + spare).astype(np.int32)
    table = np.full((R, width), -7, dtype=np.int32)
    at = 0
    for r in range(R):
        table[r, :n[r]] = perm[at:at + n[r]]
        at += n[r]
    stack = np.full(sum(n) + spare if room is None else room, -9, dtype=np.int32)
    stack[:spare] = perm[at:]
    return table, stack, spare


def check(dev, lens, new, held, T, page=64, width=40, spare=100, num_free=None, room=None, inplace=True, want_err=0, seed=0,
          table_cols=None):
    rng = np.random.default_rng(seed)
    table, stack, free = build(rng, lens, held, width, spare, room)
    if num_free is not None:
        free = num_free
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)  # noqa: E731
    g = {"lengths": i32(lens), "held": i32(held), "num_free": i32([free])}
    wide = torch.full((len(lens), table_cols or width), -5, dtype=torch.int32, device=dev)
    d_table = wide[:, :width]
    d_table.copy_(i32(table.reshape(len(lens), width)))
    d_stack = i32(stack)
    outs = {} if inplace else {f"{k}_out": torch.full_like(v, -3) for k, v in g.items()}
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = dsa.dsa_batch_plan(g["lengths"], i32(new), g["held"], d_table, d_stack, g["num_free"], T, page_size=page,
                             error_word=err, **outs)
    torch.cuda.synchronize()
    want, bits = S.plan(lens, new, held, table, stack, free, T, page)
    assert err.item() == bits == want_err
    for name, t in zip(NAMES, got):
        assert t.cpu().tolist() == want[name], name
    for k, v in g.items():
        if inplace:
            assert v.cpu().tolist() == want[k], k
        else:
            assert outs[f"{k}_out"].cpu().tolist() == want[k], k
            assert v.cpu().tolist() == {"lengths": list(lens), "held": list(held), "num_free": [free]}[k]
    assert np.array_equal(d_table.cpu().numpy(), table)
    assert np.array_equal(d_stack.cpu().numpy(), stack)
    if table_cols:
        assert (wide[:, width:] == -5).all()


def pages(n, page):
    return -(-max(n, 0) // page)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("page", [1, 16, 33, 64])
@pytest.mark.parametrize("R,most", [(1, 1), (1, 700), (7, 90), (33, 40), (257, 3)])
def test_steps(gpu, R, most, page, inplace):
    rng = np.random.default_rng(R + page)
    lens = rng.integers(0, 500, R)
    held = np.array([pages(int(n), page) for n in lens])
    new = rng.integers(0, most + 1, R)
    new[0] = most
    new[rng.random(R) < 0.15] = -1  # these end
    shrunk = rng.random(R) < 0.2  # these were evicted
    lens[shrunk] //= 3
    check(gpu, lens.tolist(), new.tolist(), held.tolist(), int(new[new > 0].sum()) + 5, page, width=2000 // page + 8,
          spare=sum(pages(int(n), page) for n in new) + R, inplace=inplace, seed=page, table_cols=2000 // page + 11)


@pytest.mark.parametrize("T", [4096, 4097, 60000])
def test_many_tokens(gpu, T):
    new = [0, 1, 3000, 0, 17, 0]
    check(gpu, [5, 64, 0, 63, 128, 0], new, [1, 1, 0, 1, 2, 0], T, 16, width=4000, spare=300)
    check(gpu, [3] * 50, [T // 50] * 50, [1] * 50, T, 64, width=T // 50 // 64 + 2, spare=T // 64 + 60)


@pytest.mark.parametrize("R", [1023, 1024, 1025, 2500])
def test_more_requests_than_one_pass(gpu, R):
    rng = np.random.default_rng(R)
    lens = rng.integers(0, 60, R)
    held = np.array([pages(int(n), 8) for n in lens])
    new = rng.integers(-1, 12, R)
    lens[::7] //= 2
    for inplace in (False, True):
        check(gpu, lens.tolist(), new.tolist(), held.tolist(), int(new[new > 0].sum()), 8, width=12, spare=3 * R, inplace=inplace)


def test_refusals_for_pages(gpu):
    # 4 free and 1 given back: request 1 takes 3, request 2 wants 3, request 3 wants none, request 4 wants one
    check(gpu, [10, 0, 0, 20, 0], [-1, 40, 48, 5, 1], [1, 0, 0, 2, 0], 200, 16, spare=4,
          want_err=dsa.DEVERR_OUT_OF_PAGES)
    check(gpu, [0, 0], [1, 1], [0, 0], 8, 16, spare=0, want_err=dsa.DEVERR_OUT_OF_PAGES)


def test_refusals_for_room(gpu):
    # 10 places: 6, then 5 (refused), then 0 (no token), then 4 (6 + 5 + 4 > 10: refused as well)
    check(gpu, [3, 3, 3, 3], [6, 5, 0, 4], [1, 1, 1, 1], 10, 16, want_err=dsa.DEVERR_TOKEN_CAPACITY)
    check(gpu, [3, 3], [1, 0], [1, 1], 0, 16, want_err=dsa.DEVERR_TOKEN_CAPACITY)
    # a refused request still gives back what an eviction left over
    check(gpu, [3, 3], [9, 9], [5, 4], 10, 16, want_err=dsa.DEVERR_TOKEN_CAPACITY)


def test_refusals_for_width(gpu):
    check(gpu, [60, 10], [5, 5], [4, 1], 64, 16, width=4, want_err=dsa.DEVERR_INDEX_OUT_OF_RANGE)
    check(gpu, [2 ** 31 - 1, 10], [1, 5], [4, 1], 64, 1 << 30, width=4, want_err=dsa.DEVERR_INDEX_OUT_OF_RANGE)
    check(gpu, [1, 0, 4, 0], [9, 9, 9, 9], [0, 0, 1, 0], 25, 4, width=3, spare=8,
          want_err=BAD | dsa.DEVERR_OUT_OF_PAGES | dsa.DEVERR_TOKEN_CAPACITY)  # 4 + 9 positions are four pages of three


def test_inconsistent_state_is_bounded(gpu):
    check(gpu, [-5, 30, 30], [3, 3, 0], [-2, 99, 0], 16, 16, width=6, spare=9)
    check(gpu, [100, 5], [-1, 1], [7, 1], 4, 16, spare=3, room=5, want_err=dsa.DEVERR_SLOT_OUT_OF_RANGE)
    check(gpu, [5], [100], [1], 100, 16, spare=3, num_free=99,
          want_err=dsa.DEVERR_OUT_OF_PAGES)  # the stack holds four at most, six are wanted
    check(gpu, [5], [1], [1], 4, 16, spare=3, num_free=-4)
    check(gpu, [5], [20], [1], 20, 16, spare=3, num_free=-4, want_err=dsa.DEVERR_OUT_OF_PAGES)


def test_a_page_below_zero_has_no_slot(gpu):
    check(gpu, [0, 4], [5, 40], [0, 1], 50, 16, spare=2, num_free=8, room=10)  # -9 is taken from the stack


def test_nothing_to_do(gpu):
    check(gpu, [], [], [], 6, 16, width=3)
    check(gpu, [], [], [], 0, 16, width=3)
    check(gpu, [0, 0], [0, 0], [0, 0], 3, 16, width=0, spare=0)
    check(gpu, [0, 0], [1, 0], [0, 0], 3, 16, width=0, spare=4, want_err=dsa.DEVERR_INDEX_OUT_OF_RANGE)


def test_graph_replays_follow_the_state(gpu):
    """A captured step run again and again: lengths, pages and slots go on from where they are."""
    rng = np.random.default_rng(4)
    R, page, width, T = 40, 8, 60, 128
    table, stack, free = build(rng, [0] * R, [0] * R, width, 2000)
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=gpu)  # noqa: E731
    lens, held, nfree, new = i32([0] * R), i32([0] * R), i32([free]), i32([0] * R)
    d_table, d_stack = i32(table), i32(stack)
    state = {"lengths": [0] * R, "held": [0] * R, "num_free": [free]}
    dsa.dsa_batch_plan(lens, new, held, d_table, d_stack, nfree, T, page_size=page)  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dsa.dsa_batch_plan(lens, new, held, d_table, d_stack, nfree, T, page_size=page)
    for step in range(12):
        add = rng.integers(-1, 5, R)
        new.copy_(i32(add))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = S.plan(state["lengths"], add, state["held"], table, stack, state["num_free"][0], T, page)
        for name, t in zip(NAMES, got):
            assert t.cpu().tolist() == want[name], (step, name)
        state = want
        assert lens.cpu().tolist() == want["lengths"] and nfree.cpu().tolist() == want["num_free"]
        assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_stack.cpu().numpy(), stack)


@pytest.mark.parametrize("R,T,most", [(300, 2000, 6), (300, 20000, 60), (1500, 9000, 5)])
def test_graph_of_large_steps(gpu, R, T, most):
    """The same where a cluster moves the pages, where the tokens have a launch of their own, and where the
    requests take several passes, in place."""
    rng = np.random.default_rng(R)
    page, width = 4, 100
    table, stack, free = build(rng, [0] * R, [0] * R, width, 30 * R)
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=gpu)  # noqa: E731
    lens, held, nfree, new = i32([0] * R), i32([0] * R), i32([free]), i32([0] * R)
    d_table, d_stack = i32(table), i32(stack)
    state = {"lengths": [0] * R, "held": [0] * R, "num_free": [free]}
    dsa.dsa_batch_plan(lens, new, held, d_table, d_stack, nfree, T, page_size=page)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dsa.dsa_batch_plan(lens, new, held, d_table, d_stack, nfree, T, page_size=page)
        tail = got[3] + 1  # what follows in the stream sees the tokens
    for step in range(6):
        add = rng.integers(-1, most + 1, R)
        if step > 2:
            shrunk = rng.random(R) < 0.3
            now = np.where(shrunk, np.array(state["lengths"]) // 2, state["lengths"])
            state["lengths"] = now.tolist()
            lens.copy_(i32(now))
        new.copy_(i32(add))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = S.plan(state["lengths"], add, state["held"], table, stack, state["num_free"][0], T, page)
        for name, t in zip(NAMES, got):
            assert t.cpu().tolist() == want[name], (step, name)
        assert torch.equal(tail, got[3] + 1)
        state = want
        assert lens.cpu().tolist() == want["lengths"] and held.cpu().tolist() == want["held"]
        assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_stack.cpu().numpy(), stack)


def test_two_plans_at_once(gpu):
    """Two batches of their own, on two streams."""
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=gpu)  # noqa: E731
    rng = np.random.default_rng(7)
    streams, runs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s in range(2):
        R = 400
        lens, new = rng.integers(0, 900, R), rng.integers(-1, 30, R)
        held = [pages(int(n), 8) for n in lens]
        table, stack, free = build(rng, lens, held, 140, 4 * R)
        runs.append((lens, new, held, table, stack, free, [i32(lens), i32(new), i32(held), i32(table), i32(stack), i32([free])]))
    torch.cuda.synchronize()
    outs = []
    for (_, _, _, _, _, _, d), st in zip(runs, streams):
        with torch.cuda.stream(st):
            outs.append(dsa.dsa_batch_plan(*d, 12000, page_size=8))
    torch.cuda.synchronize()
    for (lens, new, held, table, stack, free, d), got in zip(runs, outs):
        want, bits = S.plan(lens, new, held, table, stack, free, 12000, 8)
        assert bits == 0
        for name, t in zip(NAMES, got):
            assert t.cpu().tolist() == want[name], name
        assert np.array_equal(d[3].cpu().numpy(), table) and np.array_equal(d[4].cpu().numpy(), stack)


def test_side_stream_and_given_outputs(gpu):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    outs = {"cu_tokens": i32([-1] * 3), "req_of_token": i32([-1] * 4), "positions": i32([-1] * 4),
            "token_lengths": i32([-1] * 4), "out_loc": torch.full((4,), -2, device=gpu)}
    lens, new, held, table, stack, nf = i32([5, 0]), i32([2, 1]), i32([1, 0]), i32([[3, 0], [0, 0]]), i32([1, 4]), i32([2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dsa.dsa_batch_plan(lens, new, held, table, stack, nf, 4, page_size=16, **outs)
    side.synchronize()
    assert all(a is b for a, b in zip(got, outs.values()))
    assert outs["out_loc"].tolist() == [3 * 16 + 5, 3 * 16 + 6, 4 * 16, -1] and outs["cu_tokens"].tolist() == [0, 2, 3]


def test_binding_refusals(gpu):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)  # noqa: E731
    ok = dict(lengths=i32([1, 1]), new_tokens=i32([1, 1]), held=i32([1, 1]), block_table=i32([[0], [1]]),
              free_pages=i32([2]), num_free=i32([1]), tokens=2, page_size=16)
    for name, bad in [("held", i32([1])), ("new_tokens", None), ("num_free", i32([1, 1])), ("tokens", -1),
                      ("block_table", i32([[0]])), ("free_pages", i32([[2]])), ("lengths", i32([1, 1]).long()),
                      ("held", torch.ones(2, dtype=torch.int32))]:
        with pytest.raises(ValueError):
            dsa.dsa_batch_plan(**{**ok, name: bad})
    with pytest.raises(ValueError):
        dsa.dsa_batch_plan(**ok, out_loc=torch.zeros(3, dtype=torch.int64, device=gpu))
    with pytest.raises(dsa.DsaError):
        dsa.dsa_batch_plan(**{**ok, "page_size": 0})
