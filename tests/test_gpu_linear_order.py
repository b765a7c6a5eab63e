"""Weights that are written on the stream just before the product that reads them:
laid out anew in the same buffer, changed in place by a kernel of torch, or copied by
a kernel of the library that lets its successor start while it still writes
(csa2_paged_reorder, whose pages are any bytes). The product has to see all of them,
whichever of its forms the sizes choose.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

PER = {"e8m0": 32, "e4m3": 16}
# terms made by the product, in one CTA and in clusters; terms ahead, clusters and single CTAs; runs; bf16 values, whole and
# in clusters
SHAPES = [(1, 256, 40), (1, 4096, 640), (2, 2048, 1000), (3, 1024, 520), (8, 2048, 700), (12, 512, 6000), (9, 96, 40000), (20, 288, 20000),
          (80, 1024, 300), (130, 512, 20000)]


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


def two_matrices(csa2, g, shape, form):
    T, n_in, n_out = shape
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    packed = []
    for _ in range(2):
        data = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale = torch.randint(40, 60, (n_out, n_in // PER[form]), generator=g, device="cuda", dtype=torch.uint8)
        packed.append((data, scale + 80 if form == "e8m0" else scale))
    ws = csa2.fp4_linear_workspace(T, n_in, form)
    laid = [csa2.fp4_weights(*p, form) for p in packed]
    want = []
    for w in laid:
        torch.cuda.synchronize()
        want.append(torch.empty(T, n_out, device="cuda"))
        csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=want[-1])
    torch.cuda.synchronize()
    assert not torch.equal(*want)
    return x, ws, packed, laid, want


@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("shape", SHAPES)
def test_weights_laid_out_or_changed_just_before(csa2, shape, form):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x, ws, packed, laid, want = two_matrices(csa2, g, shape, form)
    w, change = laid[0].clone(), laid[0] ^ laid[1]
    outs = [torch.zeros_like(want[0]) for _ in range(12)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        if i < 6:
            csa2.csa2_fp4_weights(*packed[i % 2], w, form)
        else:  # it holds the second
            torch.bitwise_xor(w, change, out=w)
        csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 2]), i
    assert csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("shape", SHAPES)
def test_weights_behind_a_kernel_that_lets_its_successor_start(csa2, shape, form, captured):
    g = torch.Generator(device="cuda").manual_seed(sum(shape) + 1)
    x, ws, _, laid, want = two_matrices(csa2, g, shape, form)
    entries = laid[0].numel() // 256
    assert laid[0].numel() % 256 == 0
    page = 16
    while page <= entries:
        page *= 2
    # pages 0 and 1 hold the matrices, page 2 the weights in use: a copy of either
    pool, scales = torch.zeros(3, page, 256, dtype=torch.uint8, device="cuda"), torch.zeros(3, page, 32, dtype=torch.uint8, device="cuda")
    for p, w in zip(pool, laid):
        p.view(-1)[:w.numel()] = w
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    parents, fresh, table, n = [ints(0, 0), ints(1, 1)], ints(-1, 2), ints(0, 1).view(2, 1), ints(entries, entries)
    table_out, n_out = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), ints(0, 0)
    w = pool[2].view(-1)[:laid[0].numel()]
    outs = [torch.zeros_like(want[0]) for _ in range(6)]

    def go():
        for i, out in enumerate(outs):
            csa2.csa2_paged_reorder(parents[i % 2], fresh, table, n, table_out, n_out, kv_data=pool, kv_scale=scales)
            csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        graph.replay()
    else:
        go()
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 2]), i
    assert table_out.view(-1).tolist() == [1, 2] and csa2.csa2_get_last_error() == 0
