"""A whole serving step (plan, norms with rotation by place and cache write, means, scores, choice,
attention with a distance bias) captured once and replayed, against the same calls made one by one: bit for
bit, over prompts, decode, evictions between the replays, ends, and two such graphs in turn."""
import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa

pytestmark = pytest.mark.gpu

BF16, FP8 = dsa.CACHE_BF16, dsa.CACHE_FP8_SCALED
R, H, PAGE, WIDTH, POOL, T, K = 5, 8, 16, 16, 64, 96, 4


class Batch:
    def __init__(self, dev, kind):
        i32 = dict(dtype=torch.int32, device=dev)
        self.dev, self.kind = dev, kind
        row = 264 if kind == FP8 else 256
        self.cache = torch.zeros((POOL * PAGE, row), dtype=torch.uint8 if kind == FP8 else torch.bfloat16, device=dev)
        self.summary = torch.zeros((POOL, 256), dtype=torch.bfloat16, device=dev)
        self.lens, self.held, self.seen, self.new = (torch.zeros(R, **i32) for _ in range(4))
        self.table, self.kpos = torch.full((R, WIDTH), -1, **i32), torch.zeros((R, WIDTH * PAGE), **i32)
        self.free, self.nfree = torch.arange(POOL, **i32), torch.full((1,), POOL, **i32)
        self.mass, self.err = torch.zeros((R, WIDTH * PAGE), device=dev), torch.zeros(1, **i32)
        self.q, self.k = (torch.zeros(s, dtype=torch.bfloat16, device=dev) for s in ((T, H, 256), (T, 256)))
        self.w = torch.full((256,), 1.25, dtype=torch.bfloat16, device=dev)
        self.weights = torch.linspace(0.1, 1.0, T * H, device=dev).view(T, H)
        self.slopes = torch.tensor([2.0 ** -i for i in range(H)], device=dev)

    def step(self):
        cu, req, pos, tlen, loc, place = dsa.dsa_batch_plan(
            self.lens, self.new, self.held, self.table, self.free, self.nfree, T, page_size=PAGE, error_word=self.err,
            seen=self.seen, key_positions=self.kpos)
        x = dsa.dsa_qk_norm_rope(self.q, self.k, place, None, 1e-6, self.cache, self.kind, loc, q_norm=256, k_norm=256,
                                 q_weight=self.w, k_weight=self.w, q_out=torch.zeros_like(self.q), error_word=self.err)
        dsa.dsa_block_pool(self.cache, self.kind, self.table, pos, self.lens, self.summary, page_size=PAGE, req_of_token=req,
                           error_word=self.err)
        scores = dsa.dsa_block_scores(x, self.summary, self.table, tlen, 1 / 16, page_size=PAGE, req_of_token=req,
                                      weights=self.weights, error_word=self.err)
        blocks, own, own_len = dsa.dsa_block_select(scores, self.table, tlen, K, page_size=PAGE, req_of_token=req, sink=1,
                                                    recent=2, error_word=self.err)
        out = dsa.dsa_paged_attn(x, self.cache, self.kind, own, own_len, 1 / 16, page_size=PAGE, error_word=self.err)
        biased = dsa.dsa_paged_attn(x, self.cache, self.kind, self.table, tlen, 1 / 16, page_size=PAGE, req_of_token=req,
                                    slopes=self.slopes, q_positions=place, key_positions=self.kpos, error_word=self.err)
        return cu, req, pos, tlen, loc, place, x, scores, blocks, own, own_len, out, biased

    def evict(self, budget, seed):
        self.mass.copy_(torch.rand(self.mass.shape, generator=torch.Generator(device=self.dev).manual_seed(seed), device=self.dev))
        dsa.dsa_cache_evict(self.cache, self.kind, self.table, self.lens, self.mass, budget, page_size=PAGE, sink=1, recent=4,
                            positions=self.kpos, error_word=self.err)
        left = self.lens.tolist()
        pos = torch.tensor([p for n in left for p in range(n)], dtype=torch.int32, device=self.dev)
        req = torch.tensor([r for r, n in enumerate(left) for _ in range(n)], dtype=torch.int32, device=self.dev)
        dsa.dsa_block_pool(self.cache, self.kind, self.table, pos, self.lens, self.summary, page_size=PAGE, req_of_token=req,
                           error_word=self.err)

    def state(self):
        return [self.cache, self.summary, self.lens, self.held, self.seen, self.table, self.kpos, self.free, self.nfree]


STEPS = [[40, 0, 17, 0, 39], [1, 1, 1, 60, 1], [1, 1, 1, 1, 1], 20, [1, 30, 1, 1, 1], [1, 1, -1, 1, 0], [1, 1, 90, 1, 1], 33,
         [1, 1, 1, 1, 1], [-1, -1, -1, -1, -1], [0, 0, 0, 0, 0], [20, 20, 20, 16, 20]]


@pytest.mark.parametrize("kind", [BF16, FP8])
def test_replays_of_a_whole_step(gpu, kind):
    eager, captured = [Batch(gpu, kind) for _ in range(2)], [Batch(gpu, kind) for _ in range(2)]
    captured[0].step()  # loads the kernels: no request, no token
    torch.cuda.synchronize()
    graphs = []
    for b in captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = b.step()
        graphs.append((g, got))
    gen = torch.Generator(device=gpu).manual_seed(5)
    for n, step in enumerate(STEPS):
        if isinstance(step, int):
            for b in eager + captured:
                b.evict(step, n)
            continue
        for e, c, (g, got), new in zip(eager, captured, graphs, (step, step[::-1])):
            q = torch.randn((T, H, 256), generator=gen, device=gpu).to(torch.bfloat16)
            k = torch.randn((T, 256), generator=gen, device=gpu).to(torch.bfloat16)
            for b in (e, c):
                b.q.copy_(q)
                b.k.copy_(k)
                b.new.copy_(torch.tensor(new, dtype=torch.int32))
            want = e.step()
            g.replay()
            torch.cuda.synchronize()
            assert e.err.item() == c.err.item() == 0
            for i, (a, b) in enumerate(zip(want, got)):
                assert torch.equal(a, b), (n, i)
            for i, (a, b) in enumerate(zip(e.state(), c.state())):
                assert torch.equal(a, b), (n, "state", i)
            tokens = want[0][-1].item()
            assert tokens == sum(max(m, 0) for m in new)
            assert (want[-1][:tokens] != 0).any(2).all() and (want[-2][:tokens] != 0).any(2).all()
            assert (want[-1][tokens:] == 0).all() and (want[-2][tokens:] == 0).all()
