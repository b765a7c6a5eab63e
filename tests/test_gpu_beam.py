"""Beam selection and reordering (csa2_beam_select, csa2_paged_reorder,
csa2_reorder_rows) against the definition in 64 bits.

Tolerance of a log sum. A term 2^a, a <= 0, is off by 2^-22 (the exponential) and by
|a| ln 2 times 2^-23 (two roundings of its argument); weighted by the terms
themselves |a| ln 2 averages to at most log V < 16: 2^-22 + 2^-19. A thread adds at
most V / 1024 + 32 terms one after another to each of four sums, and every value
passes at most 40 further operations: (V / 1024 + 80) 2^-24. Together below
(V / 1024 + 160) 2^-23 = tol(V), relative to the sum, absolute in its logarithm. A
score is x - lse + score in 64 bits, rounded once: tol(V) + 2^-24 |score|.

Order: by x within a row, exactly (W = 1 is compared for equality); between rows
candidates closer than 2 tol(V) may change places.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tol(V):
    return (V / 1024 + 160) * 2.0 ** -23


def reference(x, scores):
    """All candidates' scores [B, W * V] in 64 bits, -inf where there is none."""
    xd = x.double()
    lse = torch.logsumexp(xd, -1)
    # (x - lse as x less the row's largest, less the log of what is left: of n equal values -log n, which the sum of the
    # type's lowest value and a logarithm loses in 64 bits too)
    top = xd.amax(-1, keepdim=True)
    s = (xd - top) - torch.log(torch.exp(xd - top).sum(-1, keepdim=True)) + (0 if scores is None else scores.double()[..., None])
    bad = ~torch.isfinite(lse)
    if scores is not None:
        bad |= ~torch.isfinite(scores)
    s = torch.where(bad[..., None] | (xd == -INF), torch.full_like(s, -INF), s)
    return s.flatten(1), lse


def call(csa2, x, scores, k, with_lse=True):
    B, W, V = x.shape
    o = (torch.full((B, k), 7.0, device="cuda"), torch.full((B, k), 7, dtype=torch.int32, device="cuda"),
         torch.full((B, k), 7, dtype=torch.int32, device="cuda"))
    lse = torch.full((B, W), 7.0, device="cuda") if with_lse else None
    csa2.csa2_beam_select(x, scores, *o, csa2.beam_select_workspace(B, W, V, k), lse=lse)
    return (*o, lse)


def check(x, scores, got):
    B, W, V = x.shape
    out, parents, tokens, lse = got
    k = out.shape[1]
    s, ref_lse = reference(x, scores)
    t = tol(V)
    fine = torch.isfinite(ref_lse)
    if lse is not None:
        assert ((lse.double() - ref_lse).abs()[fine] <= t + 2.0 ** -23 * ref_lse.abs()[fine]).all()
    first = torch.arange(B, device="cuda")[:, None] * W
    best, _ = torch.sort(s, descending=True, stable=True)
    n = (best > -INF).sum(1).clamp(max=k)
    col = torch.arange(k, device="cuda")[None]
    live = col < n[:, None]
    assert torch.equal(parents >= 0, live) and torch.equal(tokens >= 0, live) and (out[~live] == -INF).all()
    assert (parents[~live] == -1).all() and (tokens[~live] == -1).all()
    place = ((parents - first) * V + tokens).long()
    assert ((parents - first)[live] < W).all() and (tokens[live] < V).all()
    best = torch.nn.functional.pad(best, (0, max(0, k - best.shape[1])), value=-INF)[:, :k]
    mine = s.gather(1, torch.where(live, place, torch.zeros_like(place)))
    assert ((mine - best).abs()[live] <= 2 * t).all()
    assert ((out.double() - mine).abs()[live] <= t + 2.0 ** -23 * mine.abs()[live]).all()
    for b in range(B):
        p = place[b][live[b]].tolist()
        assert len(set(p)) == len(p)
        # within a row: by logit, then by place
        xs = x[b].flatten().double()
        by_row = {}
        for q in p:
            by_row.setdefault(q // V, []).append((-float(xs[q]), q))
        for w, c in by_row.items():
            assert c == sorted(c)
            if len(c) < k:  # nothing better of the row is left out
                row = x[b, w].double().clone()
                row[[q % V for _, q in c]] = -INF
                left = row.argmax()
                if row[left] > -INF and len(p) == k:
                    assert float(s[b, w * V + left]) <= float(mine[b][live[b]][-1]) + 2 * t


def make(kind, g, B, W, V, dtype):
    if kind == "normal":
        x = torch.randn(B, W, V, generator=g, device="cuda") * 3
    elif kind == "equal":
        x = torch.full((B, W, V), 1.5, device="cuda")
    elif kind == "few":  # few different values: ties everywhere
        x = torch.randint(-2, 3, (B, W, V), generator=g, device="cuda").float()
    elif kind == "rising":
        x = torch.arange(V, device="cuda").float().expand(B, W, V) * (8.0 / V)
    elif kind == "falling":
        x = -torch.arange(V, device="cuda").float().expand(B, W, V) * (8.0 / V)
    elif kind == "masked":  # hardly anything may follow
        x = torch.randn(B, W, V, generator=g, device="cuda")
        x = x.masked_fill(torch.rand(B, W, V, generator=g, device="cuda") < 1 - 3.0 / V, -INF)
    elif kind == "lowest":
        x = torch.randn(B, W, V, generator=g, device="cuda")
        x = x.masked_fill(torch.rand(B, W, V, generator=g, device="cuda") < 0.9, torch.finfo(dtype).min)
        x[:, 0] = torch.finfo(dtype).min
    elif kind == "tiny":  # closer than any sum with their log sum can tell
        x = torch.randn(B, W, V, generator=g, device="cuda") * 10.0 ** torch.randint(-20, -8, (B, W, 1), generator=g, device="cuda")
    elif kind == "peaked":
        x = torch.randn(B, W, V, generator=g, device="cuda")
        x[..., V // 2] = 60.0
    else:
        x = torch.randn(B, W, V, generator=g, device="cuda") * 1e4
    return x.to(dtype).contiguous()


KINDS = ["normal", "equal", "few", "rising", "falling", "masked", "lowest", "peaked", "wide", "tiny"]
SIZES = [(1, 1, 1, 1), (2, 3, 2, 4), (1, 4, 7, 8), (3, 2, 33, 5), (2, 8, 1000, 16), (1, 4, 5003, 64), (40, 16, 2051, 32),
         (1, 1, 40009, 64), (2, 64, 515, 64), (1, 2, 131075, 7)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", SIZES)
def test_select(csa2, size, kind, dtype):
    B, W, V, k = size
    g = gen(B + W + V)
    x = make(kind, g, B, W, V, dtype)
    scores = -20.0 * torch.rand(B, W, generator=g, device="cuda")
    check(x, scores, call(csa2, x, scores, k))
    assert csa2.csa2_get_last_error() == 0


# rows in many parts, whose lists are merged in registers: two, four and sixteen to one, of up to 64 keys
PARTS = [(1, 16, 50261, 32), (4, 16, 8193, 64), (1, 3, 70001, 33), (1, 1, 600011, 17), (1, 7, 90001, 5), (2, 1, 500009, 64),
         (1, 2, 300007, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["normal", "few", "rising", "masked", "lowest", "tiny"])
@pytest.mark.parametrize("size", PARTS)
def test_select_from_many_parts(csa2, size, kind, dtype):
    test_select(csa2, size, kind, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 5, 8, 255, 2048, 4097, 30011])
def test_rows_at_every_alignment(csa2, V, dtype):
    """Rows that begin anywhere: the values around them are larger and may not be seen."""
    g = gen(V)
    for shift in range(9):
        for more in (0, 1, 3):
            room = torch.full((3 * (V + more) + 32,), 1e4, device="cuda").to(dtype)
            x = room[shift:shift + 3 * (V + more)].view(1, 3, V + more)[..., :V]
            x.copy_(torch.randn(1, 3, V, generator=g, device="cuda"))
            check(x, None, call(csa2, x, None, 6))
    assert csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("V,k", [(50, 3), (5000, 17), (128259, 64)])
def test_likeliest_tokens_of_single_rows(csa2, V, k):
    """W = 1: exactly the stable order of the logits."""
    g = gen(k)
    x = (torch.randn(5, 1, V, generator=g, device="cuda") * 4).bfloat16()
    _, parents, tokens, _ = call(csa2, x, None, k)
    _, want = torch.sort(x[:, 0].float(), descending=True, stable=True)
    assert torch.equal(tokens.long(), want[:, :k])
    assert torch.equal(parents, torch.arange(5, dtype=torch.int32, device="cuda")[:, None].expand(5, k))


def test_equal_beams_go_by_place(csa2):
    """Rows alike with scores alike: the lower beam first, then the lower token."""
    x = torch.randint(0, 3, (1, 1, 500), generator=gen(1), device="cuda").float().expand(2, 4, 500).contiguous()
    out, parents, tokens, _ = call(csa2, x, torch.zeros(2, 4, device="cuda"), 64)
    s, _ = reference(x, None)
    want = torch.sort(s, descending=True, stable=True).indices[:, :64]
    first = torch.arange(2, device="cuda")[:, None] * 4
    assert torch.equal(((parents - first) * 500 + tokens).long(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zeros_of_either_sign_are_equal(csa2, dtype):
    g = gen(2)
    x = torch.where(torch.rand(3, 2, 5003, generator=g, device="cuda") < 0.5, 0.0, -0.0).to(dtype)
    x[..., ::7] = -1.0
    check(x, torch.zeros(3, 2, device="cuda"), call(csa2, x, torch.zeros(3, 2, device="cuda"), 40))
    _, _, tokens, _ = call(csa2, x[:, :1].contiguous(), None, 64)
    want = [i for i in range(100) if i % 7][:64]
    assert tokens.tolist() == [want] * 3


def test_beams_that_take_no_part(csa2):
    g = gen(21)
    x = torch.randn(3, 4, 3000, generator=g, device="cuda")
    scores = torch.tensor([0.0, -INF, -1.0, -INF], device="cuda").repeat(3, 1)
    x[0, 2] = -INF            # nothing may follow
    x[1, :] = -INF            # a sequence without candidates
    x[2, 0, 1:] = -INF        # an ended beam: its end token for nothing
    x[2, 0, 0] = 0.0
    got = call(csa2, x, scores, 20)
    check(x, scores, got)
    assert (got[1][0] == 0).all() and (got[1][1] == -1).all()
    assert (got[1][2][0], got[2][2][0], got[0][2][0]) == (8, 0, 0.0)
    assert csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("bad", [float("nan"), INF])
@pytest.mark.parametrize("at", [0, 2999, 1500, 3])
def test_rows_without_a_sum_are_reported(csa2, bad, at):
    g = gen(22)
    x = torch.randn(2, 3, 3000, generator=g, device="cuda")
    x[1, 1, at] = bad
    scores = torch.zeros(2, 3, device="cuda")
    got = call(csa2, x, scores, 30)
    assert csa2.csa2_get_last_error() == -7
    assert csa2.csa2_get_last_error() == 0
    clean = x.clone()
    clean[1, 1] = -INF
    want = call(csa2, clean, scores, 30)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    assert got[3][1, 1].isnan() and not (got[1] == 4).any()
    assert csa2.csa2_get_last_error() == 0


def test_select_captured_and_replayed_beside_another_stream(csa2):
    g = gen(30)
    x = torch.randn(4, 8, 20011, generator=g, device="cuda").bfloat16()
    scores = -torch.rand(4, 8, generator=g, device="cuda")
    want = call(csa2, x, scores, 16)
    ws = csa2.beam_select_workspace(4, 8, 20011, 16)
    out = [torch.empty_like(t) for t in want[:3]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.csa2_beam_select(x, scores, *out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(csa2, x, scores, 16)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, out, other):
        assert torch.equal(a, b) and torch.equal(a, c)


# ---- states ----------------------------------------------------------------------

WIDTHS = (("kv_data", 256), ("kv_scale", 32), ("ik_data", 64), ("ik_scale", 4))


def pool(g, layers, pages, page):
    return {name: torch.randint(0, 256, (layers, pages, page, w), generator=g, device="cuda", dtype=torch.uint8)
            for name, w in WIDTHS}


def reorder_by_hand(parents, fresh, table, counts, table_out, n_out, planes, page):
    planes = {k: v.clone() for k, v in planes.items()}
    before = {k: v.clone() for k, v in planes.items()}
    table_out, n_out, seen = table_out.clone(), n_out.clone(), set()
    for r, p in enumerate(parents):
        if p == -1:
            n_out[r] = 0
            continue
        n = counts[p]
        n_out[r] = n
        used = -(-n // page)
        table_out[r, :used] = table[p, :used]
        if n % page and p in seen:
            table_out[r, used - 1] = fresh[r]
            for k in planes:
                planes[k][:, fresh[r], :n % page] = before[k][:, int(table[p, used - 1]), :n % page]
        seen.add(p)
    return table_out, n_out, planes


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("layers,lens,parents", [
    (1, [5], [0, 0, 0]),                                        # a fork
    (2, [0, 1, 63, 64, 65, 200, 777, 256], [1, 1, 6, 6, 6, 4, 3, 3]),
    (3, [100, 100, 100], [2, 0, 0, -1, 2]),                     # more rows than before, one empty
    (1, [300, 17, 33, 511], [3, 2]),                            # fewer
    (2, [130] * 40, [i // 3 for i in range(40)])])
def test_reorder(csa2, page, layers, lens, parents):
    g = gen(len(parents) + page)
    R, rows = len(parents), len(lens)
    places = max(-(-n // page) for n in lens) + 2
    need = sum(-(-n // page) for n in lens)
    pages = need + R + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.randint(-5, 2 * pages, (rows, places), generator=g, device="cuda", dtype=torch.int32)  # unused places: anything
    at = 0
    for i, n in enumerate(lens):
        k = -(-n // page)
        table[i, :k] = order[at:at + k]
        at += k
    fresh = order[need:need + R].clone()
    planes = pool(g, layers, pages, page)
    table_out = torch.full((R, places), 123, dtype=torch.int32, device="cuda")
    n_out = torch.full((R,), 99, dtype=torch.int32, device="cuda")
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = reorder_by_hand(parents, fresh.tolist(), table, lens, table_out, n_out, planes, page)
    csa2.csa2_paged_reorder(torch.tensor(parents, dtype=torch.int32, device="cuda"), fresh, table, counts, table_out, n_out, **planes)
    assert csa2.csa2_get_last_error() == 0
    assert torch.equal(table_out, want[0]) and torch.equal(n_out, want[1])
    for name, _ in WIDTHS:
        assert torch.equal(planes[name], want[2][name]), name


def test_reorder_of_latents_alone_and_without_layers(csa2):
    g = gen(41)
    planes = pool(g, 1, 12, 16)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    counts = torch.tensor([20, 7], dtype=torch.int32, device="cuda")
    parents = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([8, 9, 10, 11], dtype=torch.int32, device="cuda")
    keys = planes["ik_data"].clone()
    out, n = torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_reorder(parents, fresh, table, counts, out, n, kv_data=planes["kv_data"][0], kv_scale=planes["kv_scale"][0])
    assert out.tolist() == [[0, 1], [0, 9], [2, -1], [11, -1]] and n.tolist() == [20, 20, 7, 7]
    assert torch.equal(planes["kv_data"][0, 9, :4], planes["kv_data"][0, 1, :4])
    assert torch.equal(planes["kv_scale"][0, 11, :7], planes["kv_scale"][0, 2, :7])
    assert torch.equal(planes["ik_data"], keys)


def test_reorder_reports_what_it_cannot_follow(csa2):
    g = gen(42)
    planes = pool(g, 1, 8, 16)
    before = {k: v.clone() for k, v in planes.items()}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, counts = ints([[0, 1], [2, 99], [3, 4], [5, 6]]), ints([20, 20, 33, -1])

    def go(parents, fresh):
        out, n = torch.full((len(parents), 2), 77, dtype=torch.int32, device="cuda"), torch.full((len(parents),), 55,
                                                                                                dtype=torch.int32, device="cuda")
        csa2.csa2_paged_reorder(ints(parents), ints(fresh), table, counts, out, n, **planes)
        status = csa2.csa2_get_last_error()
        for k in planes:
            assert torch.equal(planes[k], before[k])
        return status, out.tolist(), n.tolist()

    assert go([0, 4, -2, 1], [-1] * 4) == (-7, [[0, 1], [77, 77], [77, 77], [2, 99]], [20, 55, 55, 20])  # no such rows
    assert go([2, 3], [7, 7]) == (-7, [[77, 77], [77, 77]], [55, 55])       # counts past the table, below 0
    assert go([0, 0], [7, 8]) == (-7, [[0, 1], [0, -1]], [20, 20])          # a fresh page outside the pool
    assert go([1, 1], [7, 7]) == (-7, [[2, 99], [2, -1]], [20, 20])         # a page to copy that is not there
    assert go([-1], [-1]) == (0, [[77, 77]], [0])


@pytest.mark.parametrize("shape,dtype", [((4, 128, 512), torch.uint8), ((1,), None), ((16,), torch.uint8), ((3, 40), torch.float32),
                                         ((7, 4097, 16), torch.bfloat16)])
def test_reorder_rows(csa2, shape, dtype):
    if dtype is None:
        shape, dtype = (4,), torch.float32
    g = gen(50)
    src = torch.randint(0, 100, (6, *shape), generator=g, device="cuda").to(dtype)
    parents = torch.tensor([5, 0, 0, -1, 3, 3, 3, 1], dtype=torch.int32, device="cuda")
    dst = torch.full((8, *shape), 101, device="cuda").to(dtype)
    csa2.csa2_reorder_rows(src, parents, dst)
    assert csa2.csa2_get_last_error() == 0
    for r, p in enumerate(parents.tolist()):
        assert torch.equal(dst[r], src[p] if p >= 0 else torch.full_like(dst[r], 101))
    parents[2], parents[4] = 6, -2
    dst.fill_(101)
    csa2.csa2_reorder_rows(src, parents, dst)
    assert csa2.csa2_get_last_error() == -7
    assert (dst[2] == 101).all() and (dst[4] == 101).all() and torch.equal(dst[7], src[1])


def test_arguments_that_are_missing(csa2):
    f = lambda *n: torch.empty(*n, device="cuda")
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")
    calls = [(csa2.csa2_beam_select, dict(logits=f(2, 3, 40), out_scores=f(2, 4), out_parents=i(2, 4), out_tokens=i(2, 4),
                                          workspace=csa2.beam_select_workspace(2, 3, 40, 4)), dict(scores=f(2, 3))),
             (csa2.csa2_paged_reorder, dict(parents=i(2), fresh_pages=i(2), page_table=i(3, 2), n_visible=i(3),
                                            page_table_out=i(2, 2), n_visible_out=i(2),
                                            kv_data=torch.zeros(4, 16, 256, dtype=torch.uint8, device="cuda"),
                                            kv_scale=torch.zeros(4, 16, 32, dtype=torch.uint8, device="cuda")), {}),
             (csa2.csa2_reorder_rows, dict(src=f(2, 4), dst=f(3, 4), parents=i(3)), {})]
    for call_of, good, more in calls:
        call_of(**good, **more)
        for name in good:
            with pytest.raises(ValueError):
                call_of(**{**good, **more, name: None})
    csa2.csa2_get_last_error()


def test_refusals_of_the_binding(csa2):
    x = torch.zeros(2, 3, 40, device="cuda")
    s = torch.zeros(2, 3, device="cuda")
    f = lambda *n: torch.empty(*n, device="cuda")
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")
    good = dict(logits=x, scores=s, out_scores=f(2, 4), out_parents=i(2, 4), out_tokens=i(2, 4),
                workspace=csa2.beam_select_workspace(2, 3, 40, 4))
    csa2.csa2_beam_select(**good)
    for bad in (dict(logits=x.double()), dict(logits=x.cpu()), dict(logits=x[..., ::2]), dict(logits=x[:, :2]),
                dict(logits=x[:1, :1].expand(2, 3, 40)), dict(scores=f(3, 2)), dict(out_tokens=i(2, 5)),
                dict(out_parents=f(2, 4)), dict(out_scores=f(3, 4)), dict(workspace=f(4)), dict(lse=f(6))):
        with pytest.raises((ValueError, csa2.Csa2Error)):
            csa2.csa2_beam_select(**{**good, **bad})
    with pytest.raises(csa2.Csa2Error):
        csa2.csa2_beam_select(**{**good, "workspace": good["workspace"][:64]})
    kv = torch.zeros(4, 16, 256, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(4, 16, 32, dtype=torch.uint8, device="cuda")
    good = dict(parents=i(2), fresh_pages=i(2), page_table=i(3, 2), n_visible=i(3), page_table_out=i(2, 2), n_visible_out=i(2),
                kv_data=kv, kv_scale=sc)
    csa2.csa2_paged_reorder(**good)
    for bad in (dict(kv_data=None), dict(kv_data=None, kv_scale=None), dict(kv_scale=sc[:2]), dict(page_table_out=i(2, 3)),
                dict(n_visible=i(2)), dict(fresh_pages=i(3)), dict(parents=i(2).long())):
        with pytest.raises(ValueError):
            csa2.csa2_paged_reorder(**{**good, **bad})
    same = dict(good, parents=i(3), fresh_pages=i(3), n_visible_out=i(3))
    same["page_table_out"] = same["page_table"]
    with pytest.raises(csa2.Csa2Error):
        csa2.csa2_paged_reorder(**same)
    with pytest.raises(csa2.Csa2Error):
        csa2.csa2_reorder_rows(torch.zeros(2, 9, dtype=torch.uint8, device="cuda"), i(2), torch.zeros(2, 9, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        csa2.csa2_reorder_rows(f(2, 4), i(2), f(2, 8))
    assert csa2.csa2_get_last_error() == 0
