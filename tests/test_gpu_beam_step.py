"""Beam search over a paged FP4 cache, step by step as a program runs it: products
with 4-bit weights make latents, keys, queries, outputs and logits; the beams are
selected, and pages, counts and windows follow their parents.

What has to hold after any number of steps: a beam's pages hold exactly what was
appended along its own history, its score is the sum of its tokens' log
probabilities, and its attention is that of a cache written for it alone. And what
one call writes, the next may read at once.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

DIM, PAGE = 256, 16


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """One layer over a vocabulary of V tokens."""

    def __init__(self, csa2, g, V, form):
        self.csa2, self.form = csa2, form
        self.embed = torch.randn(V, DIM, generator=g, device="cuda").bfloat16()
        self.w = {}
        for name, n_out, n_in in (("kv", 640, DIM), ("q", 64 * 512, DIM), ("o", DIM, 64 * 512), ("vocabulary", V, DIM)):
            w = (torch.randn(n_out, n_in, generator=g, device="cuda") * 4).bfloat16()
            data, scale = csa2.quant_mxfp4(w) if form == "e8m0" else csa2.pack_kv_fp4(w.view(-1, 512))
            self.w[name] = csa2.fp4_weights(data.view(n_out, -1), scale.view(n_out, -1), form), n_out, n_in

    def product(self, name, x, f32=False):
        w, n_out, n_in = self.w[name]
        out = torch.empty(x.shape[0], n_out, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        ws = self.csa2.fp4_linear_workspace(x.shape[0], n_in, self.form)
        self.csa2.csa2_fp4_linear(x, w, None if f32 else out, ws, self.form, scale=1 / (4 * n_in ** 0.5), out_f32=out if f32 else None)
        return out


@pytest.mark.parametrize("form,B,W,V", [("e8m0", 2, 3, 1003), ("e4m3", 1, 4, 518), ("e8m0", 5, 8, 2500)])
def test_beams_keep_their_histories(csa2, form, B, W, V):
    g = gen(B * W)
    R, steps, windows = B * W, 37, 2
    model = Model(csa2, g, V, form)
    places = steps // PAGE + 2
    pages = R * (steps + 2 * places)
    shape = lambda w: torch.zeros(pages, PAGE, w, dtype=torch.uint8, device="cuda")
    planes = dict(kv_data=shape(256), kv_scale=shape(32), ik_data=shape(64), ik_scale=shape(4))
    free = list(range(pages - 1, -1, -1))
    table, table_next = (torch.full((R, places), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    n, n_next = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    swa, swa_next = (torch.zeros(R, windows, 128, 512, dtype=torch.uint8, device="cuda") for _ in range(2))
    angle = torch.arange(64, device="cuda").float()[:, None] * 0.3 ** torch.arange(32, device="cuda")
    rope = torch.stack([angle.cos(), angle.sin()], -1).contiguous()
    tokens = torch.zeros(B, W, dtype=torch.int32, device="cuda")
    scores = torch.full((B, W), float("-inf"), device="cuda")
    scores[:, 0] = 0.0  # the beams are one before the first selection
    rows, histories, logs, stamps = [], [[] for _ in range(R)], [0.0] * R, [[] for _ in range(R)]
    space = csa2.paged_attn_workspace(R, R)
    for step in range(steps):
        if step % PAGE == 0:  # a new page for everyone
            table[:, step // PAGE] = ints(*[free.pop() for _ in range(R)])
        x = model.embed[tokens.view(-1).long()]
        kv = model.product("kv", x)
        csa2.csa2_paged_kv_append(kv[:, :512].contiguous(), kv[:, 512:].contiguous(), page_table=table, n_visible=n, n_visible_out=n,
                                  rope=rope, **planes)
        rows.append(kv)
        for r in range(R):
            histories[r] = histories[r] + [(step, r)]
            stamps[r] = stamps[r] + [step * R + r]
        swa[torch.arange(R), :, step % 128, :8] = ints(*[step * R + r for r in range(R)]).view(torch.uint8).view(R, 1, 4).repeat(1, windows, 2)
        q = model.product("q", x).view(R, 64, 512)
        out = torch.empty_like(q)
        csa2.csa2_paged_attn(q, planes["kv_data"], planes["kv_scale"], table, n, out, space, sm_scale=512 ** -0.5)
        h = model.product("o", out.view(R, -1))
        logits = model.product("vocabulary", h, f32=True).view(B, W, V)
        best, parents, tokens = torch.empty(B, W, device="cuda"), *(torch.empty(B, W, dtype=torch.int32, device="cuda") for _ in range(2))
        csa2.csa2_beam_select(logits, scores, best, parents, tokens, csa2.beam_select_workspace(B, W, V, W))
        fresh = ints(*[free.pop() for _ in range(R)])
        csa2.csa2_paged_reorder(parents.view(-1), fresh, table, n, table_next, n_next, **planes)
        csa2.csa2_reorder_rows(swa, parents.view(-1), swa_next)
        assert csa2.csa2_get_last_error() == 0
        log = torch.log_softmax(logits.double(), -1).view(R, V)
        p = parents.view(-1).tolist()
        assert all(b * W <= p[b * W + w] < (b + 1) * W for b in range(B) for w in range(W))
        logs = [logs[p[r]] + float(log[p[r], int(tokens.view(-1)[r])]) for r in range(R)]
        histories, stamps = [histories[i] for i in p], [stamps[i] for i in p]
        assert torch.allclose(best.view(-1).double().cpu(), torch.tensor(logs, dtype=torch.float64), rtol=1e-6, atol=1e-4)
        assert (best[:, :-1] >= best[:, 1:]).all()
        # (pages that nobody holds any more are free again)
        used = set(table_next[:, :step // PAGE + 1].flatten().tolist())
        free += [f for f in fresh.tolist() if f not in used]
        table, table_next, n, n_next, scores, swa, swa_next = table_next, table, n_next, n, best, swa_next, swa
    assert (n == steps).all()
    # each beam's entries, written for it alone in order
    alone = {k: torch.zeros(R * places, PAGE, v.shape[-1], dtype=torch.uint8, device="cuda") for k, v in planes.items()}
    own = torch.arange(R * places, dtype=torch.int32, device="cuda").view(R, places)
    kv = torch.stack([torch.stack([rows[s][r] for s, r in histories[i]]) for i in range(R)]).view(R * steps, 640)
    m = torch.zeros(R, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_kv_append(kv[:, :512].contiguous(), kv[:, 512:].contiguous(), page_table=own, n_visible=m, n_visible_out=m, rope=rope,
                              **alone)
    e = torch.arange(steps, device="cuda")
    for name in planes:
        here = planes[name][table.long()[:, e // PAGE], e % PAGE]
        there = alone[name][own.long()[:, e // PAGE], e % PAGE]
        assert torch.equal(here, there), name
    q = model.product("q", model.embed[tokens.view(-1).long()]).view(R, 64, 512)
    a, b = torch.empty_like(q), torch.empty_like(q)
    csa2.csa2_paged_attn(q, planes["kv_data"], planes["kv_scale"], table, n, a, space, sm_scale=512 ** -0.5)
    csa2.csa2_paged_attn(q, alone["kv_data"], alone["kv_scale"], own, m, b, space, sm_scale=512 ** -0.5)
    assert torch.equal(a, b)
    # each beam's windows
    for i in range(R):
        want = ints(*stamps[i]).view(torch.uint8).view(steps, 4)
        assert torch.equal(swa[i, 0, :steps, :4], want) and torch.equal(swa[i, 1, :steps, 4:8], want)
    # nobody else writes where a beam writes next
    last = table[:, (steps - 1) // PAGE].tolist()
    assert steps % PAGE == 0 or len(set(last)) == R
    assert csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("T", [3, 20, 80])
def test_attention_behind_the_product_that_made_its_queries(csa2, T):
    """The attention reads its queries before it waits for the kernel before it: a product may not let it start early."""
    g = gen(T)
    n, k = 700, 64
    w = (torch.randn(64 * 512, DIM, generator=g, device="cuda") * 4).bfloat16()
    weights = csa2.fp4_weights(*csa2.quant_mxfp4(w), "e8m0")
    kv = torch.randn(T, 768, 512, generator=g, device="cuda").bfloat16()
    data, scale = csa2.pack_kv_fp4(kv)
    n_visible = torch.full((T,), n, dtype=torch.int32, device="cuda")
    idx = torch.stack([torch.randperm(n, generator=g, device="cuda")[:k].sort().values.int() for _ in range(T)])
    swa = torch.zeros(T, 1, 32, 512, dtype=torch.uint8, device="cuda")
    ws, aws = csa2.fp4_linear_workspace(T, DIM, "e8m0"), csa2.attn_workspace(T, k, 32)
    q = torch.zeros(T, 1, 64, 512, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    xs = [torch.randn(T, DIM, generator=g, device="cuda").bfloat16() for _ in range(8)]

    def go(x, wait):
        csa2.csa2_fp4_linear(x, weights, q.view(T, -1), ws, "e8m0", scale=1 / (64 * 512 ** 0.5))
        if wait:
            torch.cuda.synchronize()
        csa2.csa2_sparse_attn_decode(q, data, scale, n_visible, idx, swa, out, aws)
        return out.clone()

    want = [go(x, True) for x in xs]
    got = [go(x, False) for _ in range(3) for x in xs]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 8])
    assert csa2.csa2_get_last_error() == 0


def test_steps_on_two_streams_at_once(csa2):
    """Products and selections of two programs side by side, each with its own workspaces."""
    g = gen(77)
    V, T = 20000, 24
    jobs = []
    for form in ("e8m0", "e4m3"):
        w = (torch.randn(V, 1024, generator=g, device="cuda") * 4).bfloat16()
        data, scale = csa2.quant_mxfp4(w) if form == "e8m0" else csa2.pack_kv_fp4(w.view(-1, 512))
        jobs.append(dict(form=form, w=csa2.fp4_weights(data.view(V, -1), scale.view(V, -1), form), stream=torch.cuda.Stream(),
                         x=torch.randn(T, 1024, generator=g, device="cuda").bfloat16(), ws=csa2.fp4_linear_workspace(T, 1024, form),
                         bs=csa2.beam_select_workspace(4, 6, V, 12), logits=torch.empty(4, 6, V, device="cuda"),
                         scores=-torch.rand(4, 6, generator=g, device="cuda")))

    def go(j):
        csa2.csa2_fp4_linear(j["x"], j["w"], None, j["ws"], j["form"], scale=0.01, out_f32=j["logits"].view(T, V))
        o = torch.empty(4, 12, device="cuda"), *(torch.empty(4, 12, dtype=torch.int32, device="cuda") for _ in range(2))
        csa2.csa2_beam_select(j["logits"], j["scores"], *o, j["bs"])
        return (j["logits"].clone(), *o)

    want = [go(j) for j in jobs]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for j in jobs:
            with torch.cuda.stream(j["stream"]):
                got.append(go(j))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for a, b in zip(o, want[i % 2]):
            assert torch.equal(a, b)
    assert csa2.csa2_get_last_error() == 0


def test_offsets_past_32_bits(csa2):
    """Weights, logits and states of more than 4 GiB: the last of them, read and written whole."""
    g = gen(5)
    n_out, n_in = 530000, 16384
    data = torch.zeros(n_out, n_in // 2, dtype=torch.uint8, device="cuda")
    scale = torch.full((n_out, n_in // 32), 127, dtype=torch.uint8, device="cuda")
    data[-200:] = torch.randint(0, 256, (200, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    data[0] = 0x22  # ones
    w = csa2.fp4_weights(data, scale, "e8m0")
    assert w.numel() > 1 << 32
    back = torch.empty(200, n_in, device="cuda")
    csa2.csa2_dequant_mxfp4(data[-200:].contiguous(), scale[-200:].contiguous(), back)
    del data, scale
    for T in (1, 9, 70):
        x = torch.randint(-8, 9, (T, n_in), generator=g, device="cuda").bfloat16()
        out = torch.empty(T, n_out, device="cuda")
        csa2.csa2_fp4_linear(x, w, None, csa2.fp4_linear_workspace(T, n_in, "e8m0"), "e8m0", out_f32=out)
        assert torch.equal(out[:, -200:].double(), x.double() @ back.double().T)
        assert torch.equal(out[:, 0].double(), x.double().sum(1)) and (out[:, 1:-200] == 0).all()
    del w, out
    W, V = 54, 40_000_003
    x = torch.zeros(1, W, V, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    x[0, -1, -5:] = torch.arange(30, 35, device="cuda").bfloat16()
    o = torch.empty(1, 8, device="cuda"), *(torch.empty(1, 8, dtype=torch.int32, device="cuda") for _ in range(2))
    lse = torch.empty(1, W, device="cuda")
    csa2.csa2_beam_select(x, None, *o, csa2.beam_select_workspace(1, W, V, 8), lse=lse)
    assert o[1][0, :5].tolist() == [W - 1] * 5 and o[2][0, :5].tolist() == [V - 1 - i for i in range(5)]
    # Rows that are alike but lie differently in memory (V is odd) add their terms in another order: their log sums, and
    # with them all their scores, differ by up to 2 tol(V) = 2 (V / 1024 + 160) 2^-23 (test_gpu_beam.py). Within a row the
    # scores are exactly equal, so whichever row comes first has its lowest tokens in order.
    rest = list(zip(o[1][0, 5:].tolist(), o[2][0, 5:].tolist()))
    assert all(p < W - 1 for p, _ in rest) and all(v == sum(p == a for a, _ in rest[:i]) for i, (p, v) in enumerate(rest))
    assert torch.allclose(lse[0, :-1].double(), torch.full((W - 1,), float(V), dtype=torch.float64, device="cuda").log(), rtol=1e-4)
    del x
    src = torch.zeros(2, (3 << 30) + 16, dtype=torch.uint8, device="cuda")
    src[1, -48:] = torch.arange(48, device="cuda").to(torch.uint8)
    dst = torch.full_like(src, 9)
    csa2.csa2_reorder_rows(src, ints(1, 1), dst)
    assert torch.equal(dst[0], src[1]) and torch.equal(dst[1], src[1])
    assert csa2.csa2_get_last_error() == 0
