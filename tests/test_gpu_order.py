"""Calls one behind another on a stream, without a wait between them, eager and captured, give what the same calls give one at a
time: kernels start before the one before them has ended, and may neither read what it still writes nor write what it still
reads. Sequences of calls over the paged cache in random order, sharing workspaces, counters and buffers."""

import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


class World:
    def __init__(self, csa2, seed):
        g, r = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

        self.B, self.L, self.T = B, L, T = r.choice([1, 3, 9, 32]), r.choice([1, 2]), r.choice([1, 1, 3])
        page, self.k, n_swa = r.choice([16, 64, 128]), r.choice([64, 512]), r.choice([16, 128])
        most = 2048 // page
        pages = B * most + 3
        self.table = torch.randperm(pages, generator=g, device="cuda").int()[:B * most].view(B, most).contiguous()
        self.planes = [torch.zeros(pages, page, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
        self.nv = torch.zeros(B, dtype=torch.int32, device="cuda")
        a = torch.arange(2048, dtype=torch.float64)[:, None] * 10000 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
        self.rope = torch.stack([a.cos(), a.sin()], -1).float().cuda().contiguous()
        csa2.csa2_paged_kv_append(normal(200 * B, 512), normal(200 * B, 128), *self.planes, self.table, self.nv, self.nv, rope=self.rope)
        self.new = [(normal(B * T, 512), normal(B * T, 128)) for _ in range(3)]
        self.q, self.q2 = normal(B * L, 64, 512, scale=0.05), normal(B * L, 64, 512, scale=0.05)
        self.dq = normal(B * T, 64, 512, scale=0.05)
        self.swa = [csa2.pack_fp8(normal(B, L, n_swa, 512)) for _ in range(2)]
        self.qi, self.qs = csa2.quant_mxfp4(normal(B, 32, 128))
        self.w = torch.rand(B, 32, generator=g, device="cuda")
        self.scores, self.counters = torch.zeros(B, 2048, device="cuda"), torch.zeros(2 * B, dtype=torch.int32, device="cuda")
        self.idx = torch.full((B, self.k), -1, dtype=torch.int32, device="cuda")
        self.spaces = [csa2.topk_workspace(B, 2048, self.k), csa2.paged_sparse_attn_workspace(B, L, self.k, n_swa),
                       csa2.paged_attn_workspace(B * T, B)]
        self.out, self.out2 = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.dense, self.dense2 = torch.zeros_like(self.dq), torch.zeros_like(self.dq)
        torch.cuda.synchronize()

    def call(self, csa2, name, i):
        cache = self.planes[0], self.planes[1], self.table, self.nv
        if name == "append":
            csa2.csa2_paged_kv_append(*self.new[i % 3], *self.planes, self.table, self.nv, self.nv, rope=self.rope, interleaved=True)
        elif name == "rope":  # in place, or into another buffer
            csa2.csa2_rope(self.q, self.rope, None, self.q2 if i % 2 else self.q, interleaved=True)
        elif name == "back":
            x = (self.dense, self.out, self.dq, self.out2)[i]
            csa2.csa2_rope(x, self.rope, None, x, inverse=True)
        elif name == "score":
            csa2.csa2_paged_index_score(self.qi, self.qs, self.w, *self.planes[2:], self.table, self.nv, self.scores,
                                        tile_counters=self.counters if i % 2 else None)
        elif name == "topk":
            csa2.csa2_topk(self.scores, self.k, self.idx, self.spaces[0], n_valid=self.nv)
        elif name == "selected":
            q, out = (self.q2, self.out2) if i % 2 else (self.q, self.out)
            shape = self.B, self.L, 64, 512
            csa2.csa2_paged_sparse_attn_decode(q.view(shape), *cache, self.idx, self.swa[i // 2], out.view(shape), self.spaces[1])
        elif name == "dense":
            csa2.csa2_paged_attn(self.dq, *cache, self.dense2 if i % 2 else self.dense, self.spaces[2], causal=i < 2)
        else:
            self.q2.copy_(self.q * 0.5)

    def results(self):
        return (*self.planes, self.nv, self.q, self.q2, self.dq, self.scores, self.counters, self.idx, self.out, self.out2, self.dense,
                self.dense2)


CALLS = "append rope rope back back score topk selected selected selected dense dense copy".split()


@pytest.mark.parametrize("seed", range(12))
def test_calls_in_any_order(csa2, seed):
    r = random.Random(1000 + seed)
    calls = [(r.choice(CALLS), r.randrange(4)) for _ in range(80)]
    alone = World(csa2, seed)
    for c in calls:
        alone.call(csa2, *c)
        torch.cuda.synchronize()
    eager, captured = World(csa2, seed), World(csa2, seed)
    for c in calls:
        eager.call(csa2, *c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            captured.call(csa2, *c)
    graph.replay()
    torch.cuda.synchronize()
    for world in (eager, captured):
        for a, b in zip(alone.results(), world.results()):
            assert torch.equal(a, b)
    assert csa2.csa2_get_last_error() == 0
