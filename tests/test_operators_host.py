"""CPU checks of the entry points around the paged cache (products with 4-bit
weights, beam selection, reordering): what is refused on the host, before
anything is enqueued, and what is nothing to do."""

import ctypes

import pytest

vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
OK, ARG, SHAPE, ALIGN, WORKSPACE = 0, -1, -2, -3, -6
P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from fp4_kv_cache_02_gb300 import _build
    lib = ctypes.CDLL(_build.build())
    lib.csa2_fp4_weights_size.argtypes, lib.csa2_fp4_weights_size.restype = [i32] * 3, sz
    lib.csa2_fp4_linear_workspace_size.argtypes, lib.csa2_fp4_linear_workspace_size.restype = [i32] * 3, sz
    lib.csa2_beam_select_workspace_size.argtypes, lib.csa2_beam_select_workspace_size.restype = [i32] * 4, sz
    lib.csa2_fp4_weights.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    lib.csa2_fp4_linear.argtypes = [vp, i32, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.csa2_beam_select.argtypes = [vp, i32, i32, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.csa2_paged_reorder.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i64, i32, vp, i32, i32, vp, vp, vp, vp]
    lib.csa2_reorder_rows.argtypes = [vp, i64, i64, vp, i32, vp, vp]
    return lib


def call(fn, order, good, **change):
    args = dict(good, **change)
    assert set(args) == set(order), set(change) - set(order)
    return fn(*[args[n] for n in order], None)


WEIGHTS = "data scale n_out n_in format weights".split()
WEIGHTS_GOOD = dict(data=P, scale=P, n_out=0, n_in=64, format=0, weights=P)


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(data=None, scale=None, weights=None), OK), (dict(format=1), OK),
    (dict(n_out=-1), ARG), (dict(n_in=-32), ARG), (dict(format=2), ARG), (dict(format=-1), ARG),
    (dict(n_out=1, data=None), ARG), (dict(n_out=1, scale=None), ARG), (dict(n_out=1, weights=None), ARG),
    (dict(n_in=0), SHAPE), (dict(n_in=48), SHAPE), (dict(n_in=(1 << 30) + 32), SHAPE), (dict(n_out=1 << 30, n_in=1 << 20), SHAPE),
    (dict(n_out=1, data=P + 8), ALIGN), (dict(n_out=1, weights=P + 8), ALIGN)])
def test_weights(lib, change, status):
    assert call(lib.csa2_fp4_weights, WEIGHTS, WEIGHTS_GOOD, **change) == status


LINEAR = "x n weights n_out n_in format scale out out_f32 ws ws_bytes".split()
LINEAR_GOOD = dict(x=P, n=2, weights=P, n_out=8, n_in=64, format=0, scale=1.0, out=P, out_f32=None, ws=P, ws_bytes=0)


@pytest.mark.parametrize("change,status", [
    ({}, WORKSPACE), (dict(ws=None, ws_bytes=1 << 40), WORKSPACE), (dict(ws=P + 128, ws_bytes=1 << 40), WORKSPACE),
    (dict(n=0), OK), (dict(n_out=0), OK), (dict(n=0, x=None, out=None, ws=None), OK),
    (dict(n=-1), ARG), (dict(n_out=-1), ARG), (dict(n_in=-1), ARG), (dict(format=7), ARG), (dict(x=None), ARG),
    (dict(weights=None), ARG), (dict(out=None), ARG), (dict(out=None, out_f32=P), WORKSPACE),
    (dict(n_in=0), SHAPE), (dict(n_in=33), SHAPE), (dict(n_in=(1 << 30) + 32), SHAPE), (dict(n=1 << 30, n_out=1 << 30), SHAPE), (dict(n=1 << 30, n_in=1 << 20), SHAPE),
    (dict(x=P + 8), ALIGN), (dict(weights=P + 8), ALIGN), (dict(out=P + 1), ALIGN), (dict(out_f32=P + 2), ALIGN)])
def test_linear(lib, change, status):
    assert call(lib.csa2_fp4_linear, LINEAR, LINEAR_GOOD, **change) == status


def test_sizes(lib):
    size = lib.csa2_fp4_weights_size
    assert size(1, 32, 0) == size(128, 256, 0) == 17408 and size(129, 257 + 31, 1) == 4 * 18432
    assert size(1 << 20, 1 << 16, 0) > 1 << 32  # past 32 bits
    assert size(1, 31, 0) == size(-1, 32, 0) == size(1, 32, 3) == 0
    ws = lib.csa2_fp4_linear_workspace_size
    assert 0 < ws(1, 256, 0) < ws(9, 256, 0) < ws(32, 256, 0) < ws(32, 512, 0) < ws(64, 512, 0) and ws(65, 256, 0) > 0 and ws(65, 32, 0) > ws(64, 32, 0)
    assert ws(0, 256, 0) == ws(1, 0, 0) == ws(1, 256, 9) == 0
    assert ws(1 << 27, 32, 0) > 1 << 32
    beam = lib.csa2_beam_select_workspace_size
    assert 0 < beam(1, 1, 10, 64) < beam(1, 1, 100000, 64) and beam(1, 1, 100000, 1) < beam(1, 1, 100000, 64)
    assert beam(0, 1, 10, 1) == beam(1, 0, 10, 1) == beam(1, 1, 10, 0) == beam(1, 1, 10, 65) == 0


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("n_in", [32, 64, 256, 4096, 32768])
def test_a_workspace_for_more_tokens_does_for_fewer(lib, n_in, kind):
    sizes = [lib.csa2_fp4_linear_workspace_size(t, n_in, kind) for t in [*range(1, 140), 1021, 4096, 100003]]
    assert sizes == sorted(sizes) and sizes[0] > 0


BEAM = "logits f32 B W V ld scores k out parents tokens lse ws ws_bytes".split()
BEAM_GOOD = dict(logits=P, f32=1, B=2, W=3, V=100, ld=100, scores=P, k=4, out=P, parents=P, tokens=P, lse=None, ws=P, ws_bytes=0)


@pytest.mark.parametrize("change,status", [
    ({}, WORKSPACE), (dict(scores=None), WORKSPACE), (dict(ws=None, ws_bytes=1 << 40), WORKSPACE),
    (dict(ws=P + 64, ws_bytes=1 << 40), WORKSPACE), (dict(B=0), OK), (dict(B=0, logits=None, out=None), OK),
    (dict(B=-1), ARG), (dict(W=-1), ARG), (dict(W=0), ARG), (dict(V=-1), ARG), (dict(V=0), ARG), (dict(ld=99), ARG), (dict(k=-1), ARG),
    (dict(f32=2), ARG), (dict(logits=None), ARG), (dict(out=None), ARG), (dict(parents=None), ARG), (dict(tokens=None), ARG),
    (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(W=65), SHAPE), (dict(B=1 << 22, W=2), SHAPE),
    (dict(logits=P + 2), ALIGN), (dict(logits=P + 2, f32=0), WORKSPACE), (dict(logits=P + 1, f32=0), ALIGN), (dict(scores=P + 2), ALIGN),
    (dict(out=P + 2), ALIGN), (dict(parents=P + 2), ALIGN), (dict(tokens=P + 2), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_beam(lib, change, status):
    assert call(lib.csa2_beam_select, BEAM, BEAM_GOOD, **change) == status


REORDER = ("parents fresh R kv_data kv_scale ik_data ik_scale layers n_pages page table rows max_pages n_visible table_out "
           "n_out").split()
REORDER_GOOD = dict(parents=P, fresh=P, R=0, kv_data=P, kv_scale=P, ik_data=P, ik_scale=P, layers=2, n_pages=8, page=64, table=P, rows=3,
                    max_pages=4, n_visible=P, table_out=P + 4096, n_out=P + 4096)


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(parents=None, fresh=None, table_out=None, n_out=None), OK),
    (dict(R=-1), ARG), (dict(rows=-1), ARG), (dict(layers=-1), ARG), (dict(n_pages=-1), ARG), (dict(page=0), ARG), (dict(max_pages=-1), ARG),
    (dict(table=None), ARG), (dict(R=1, parents=None), ARG), (dict(R=1, fresh=None), ARG), (dict(R=1, n_visible=None), ARG),
    (dict(R=1, table_out=None), ARG), (dict(R=1, n_out=None), ARG), (dict(R=1, kv_data=None), ARG), (dict(R=1, ik_scale=None), ARG),
    (dict(R=1, table_out=P), ARG), (dict(R=1, n_out=P), ARG),
    (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(layers=65535), SHAPE), (dict(n_pages=1 << 26), SHAPE),
    (dict(parents=P + 2), ALIGN), (dict(fresh=P + 2), ALIGN), (dict(table=P + 2), ALIGN), (dict(n_visible=P + 2), ALIGN),
    (dict(table_out=P + 2), ALIGN), (dict(n_out=P + 2), ALIGN), (dict(kv_data=P + 8), ALIGN), (dict(kv_scale=P + 8), ALIGN),
    (dict(ik_data=P + 8), ALIGN), (dict(ik_scale=P + 4), ALIGN)])
def test_reorder(lib, change, status):
    assert call(lib.csa2_paged_reorder, REORDER, REORDER_GOOD, **change) == status


ROWS = "src rows row_bytes parents R dst".split()
ROWS_GOOD = dict(src=P, rows=4, row_bytes=64, parents=P, R=0, dst=2 * P)


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(R=3, row_bytes=0), OK), (dict(src=None, parents=None, dst=None), OK),
    (dict(rows=-1), ARG), (dict(row_bytes=-16), ARG), (dict(R=-1), ARG), (dict(R=1, src=None), ARG), (dict(R=1, parents=None), ARG),
    (dict(R=1, dst=None), ARG), (dict(R=1, dst=P), ARG), (dict(row_bytes=24), SHAPE), (dict(R=1 << 30, row_bytes=1 << 40), SHAPE),
    (dict(src=P + 8), ALIGN), (dict(dst=P + 8), ALIGN), (dict(parents=P + 2), ALIGN)])
def test_rows(lib, change, status):
    assert call(lib.csa2_reorder_rows, ROWS, ROWS_GOOD, **change) == status
