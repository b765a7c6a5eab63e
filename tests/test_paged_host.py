"""CPU checks of the paged cache's entry points: what is refused on the host,
before anything is enqueued, and what is nothing to do."""

import ctypes

import pytest

vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
OK, ARG, SHAPE, ALIGN, WORKSPACE = 0, -1, -2, -3, -6
P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from fp4_kv_cache_02_gb300 import _build
    lib = ctypes.CDLL(_build.build())
    lib.csa2_rope.argtypes = [vp, i64, i32, i32, vp, i64, i32, vp, i32, i32, vp, vp]
    lib.csa2_paged_kv_append.argtypes = [vp, vp, i32, vp, i32, vp, i64, i32, vp, i32, vp, vp, vp, vp, i64, i32, vp, i32,
                                         vp, vp, vp]
    lib.csa2_paged_index_score.argtypes = [vp, vp, vp, i32, vp, vp, i64, i32, vp, i32, vp, i64, vp, vp, vp]
    lib.csa2_paged_sparse_attn_decode.argtypes = [vp, i32, i32, vp, vp, i64, i32, vp, i32, vp, vp, i32, vp, i32, f32, vp,
                                                  vp, vp, vp, sz, vp]
    lib.csa2_paged_attn.argtypes = [vp, i32, vp, i32, vp, vp, i64, i32, vp, i32, vp, i32, f32, vp, vp, vp, vp, sz, vp]
    lib.csa2_paged_sparse_attn_workspace_size.restype = sz
    lib.csa2_paged_sparse_attn_workspace_size.argtypes = [i32] * 4
    lib.csa2_paged_attn_workspace_size.restype = sz
    lib.csa2_paged_attn_workspace_size.argtypes = [i32] * 2
    return lib


def call(fn, order, good, **change):
    args = dict(good, **change)
    assert set(args) == set(order), set(change) - set(order)
    return fn(*[args[n] for n in order], None)


ROPE = "x n heads dim rope n_rope rope_dim positions interleaved inverse out".split()
ROPE_GOOD = dict(x=P, n=0, heads=4, dim=128, rope=P, n_rope=10, rope_dim=64, positions=P, interleaved=0, inverse=0, out=P)


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(heads=0), OK), (dict(x=None, out=None), OK), (dict(positions=None), OK),
    (dict(n=-1), ARG), (dict(n=1, x=None), ARG), (dict(n=1, out=None), ARG), (dict(rope=None), ARG), (dict(dim=0), ARG),
    (dict(heads=-1), ARG), (dict(n_rope=-1), ARG), (dict(rope_dim=-32), ARG),
    (dict(rope_dim=0), SHAPE), (dict(rope_dim=48), SHAPE), (dict(rope_dim=160), SHAPE), (dict(dim=32), SHAPE),
    (dict(dim=132), SHAPE), (dict(n=1 << 60), SHAPE),
    (dict(x=P + 8), ALIGN), (dict(out=P + 8), ALIGN), (dict(rope=P + 8), ALIGN), (dict(positions=P + 2), ALIGN)])
def test_rope(lib, change, status):
    assert call(lib.csa2_rope, ROPE, ROPE_GOOD, **change) == status


POOL = dict(n_pages=8, page=64, table=P, max_pages=4, n_visible=P)
# what every paged entry point refuses of its pool and table
POOL_BAD = [(dict(n_pages=-1), ARG), (dict(page=0), ARG), (dict(page=-64), ARG), (dict(max_pages=-1), ARG),
            (dict(table=None), ARG), (dict(B=-1), ARG), (dict(n_visible=None), ARG),
            (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(n_pages=1 << 26), SHAPE),
            (dict(table=P + 2), ALIGN), (dict(n_visible=P + 2), ALIGN)]

APPEND = ("kv ik n cu B rope n_rope rope_dim positions interleaved kv_data kv_scale ik_data ik_scale n_pages page table "
          "max_pages n_visible n_visible_out").split()
APPEND_GOOD = dict(POOL, kv=P, ik=P, n=0, cu=P, B=2, rope=P, n_rope=10, rope_dim=64, positions=None, interleaved=1,
                   kv_data=P, kv_scale=P, ik_data=P, ik_scale=P, n_visible_out=None)


@pytest.mark.parametrize("change,status", POOL_BAD + [
    (dict(B=0), OK), (dict(n=-1), ARG), (dict(n=4, kv=None), ARG), (dict(n=4, ik=None), ARG), (dict(kv_data=None), ARG),
    (dict(kv_scale=None), ARG), (dict(ik_data=None), ARG), (dict(ik_scale=None), ARG), (dict(n=3, cu=None), ARG),
    (dict(rope_dim=16), SHAPE), (dict(rope_dim=256), SHAPE), (dict(rope_dim=-1), ARG),
    (dict(kv=P + 8), ALIGN), (dict(ik=P + 8), ALIGN), (dict(cu=P + 2), ALIGN), (dict(rope=P + 4), ALIGN),
    (dict(kv_data=P + 8), ALIGN), (dict(kv_scale=P + 8), ALIGN), (dict(ik_data=P + 8), ALIGN), (dict(ik_scale=P + 4), ALIGN),
    (dict(positions=P + 1), ALIGN), (dict(n_visible_out=P + 1), ALIGN)])
def test_append(lib, change, status):
    assert call(lib.csa2_paged_kv_append, APPEND, APPEND_GOOD, **change) == status


SCORE = "q q_scale w B ik_data ik_scale n_pages page table max_pages n_visible n_pos scores counters".split()
SCORE_GOOD = dict(POOL, q=P, q_scale=P, w=P, B=2, ik_data=P, ik_scale=P, n_pos=100, scores=P, counters=P)


@pytest.mark.parametrize("change,status", POOL_BAD + [
    (dict(B=0), OK), (dict(n_pos=0), OK), (dict(n_pos=0, scores=None), OK), (dict(n_pos=-1), ARG), (dict(n_pos=257), ARG),
    (dict(q=None), ARG), (dict(q_scale=None), ARG), (dict(w=None), ARG), (dict(scores=None), ARG), (dict(ik_data=None), ARG),
    (dict(q=P + 8), ALIGN), (dict(ik_data=P + 8), ALIGN), (dict(ik_scale=P + 8), ALIGN), (dict(counters=P + 4), ALIGN)])
def test_score(lib, change, status):
    assert call(lib.csa2_paged_index_score, SCORE, SCORE_GOOD, **change) == status


SPARSE = ("q B L kv_data kv_scale n_pages page table max_pages n_visible idx k swa n_swa scale out out_f32 lse ws "
          "ws_bytes").split()
SPARSE_GOOD = dict(POOL, q=P, B=2, L=1, kv_data=P, kv_scale=P, idx=P, k=64, swa=P, n_swa=128, scale=1.0, out=P,
                   out_f32=None, lse=None, ws=P, ws_bytes=0)


@pytest.mark.parametrize("change,status", POOL_BAD + [
    ({}, WORKSPACE), (dict(ws=None, ws_bytes=1 << 40), WORKSPACE), (dict(ws=P + 16, ws_bytes=1 << 40), WORKSPACE),
    (dict(B=0), OK), (dict(L=0), ARG), (dict(k=-1), ARG), (dict(n_swa=-1), ARG), (dict(swa=None), ARG),
    (dict(idx=None), ARG), (dict(q=None), ARG), (dict(out=None), ARG), (dict(k=4097), SHAPE), (dict(n_swa=513), SHAPE),
    (dict(B=1 << 20, L=1 << 12), SHAPE), (dict(q=P + 8), ALIGN), (dict(kv_data=P + 8), ALIGN), (dict(kv_scale=P + 8), ALIGN),
    (dict(out=P + 4), ALIGN), (dict(out_f32=P + 4), ALIGN), (dict(swa=P + 8), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_sparse(lib, change, status):
    assert call(lib.csa2_paged_sparse_attn_decode, SPARSE, SPARSE_GOOD, **change) == status


DENSE = ("q n cu B kv_data kv_scale n_pages page table max_pages n_visible causal scale out out_f32 lse ws "
         "ws_bytes").split()
DENSE_GOOD = dict(POOL, q=P, n=6, cu=P, B=2, kv_data=P, kv_scale=P, causal=1, scale=1.0, out=P, out_f32=None, lse=None,
                  ws=P, ws_bytes=0)


@pytest.mark.parametrize("change,status", POOL_BAD + [
    ({}, WORKSPACE), (dict(ws=None, ws_bytes=1 << 40), WORKSPACE), (dict(ws=P + 128, ws_bytes=1 << 40), WORKSPACE),
    (dict(n=0), OK), (dict(n=0, q=None, out=None), OK), (dict(B=0), OK), (dict(n=-1), ARG), (dict(n=7, cu=None), ARG),
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(kv_data=None), ARG), (dict(kv_scale=None), ARG),
    (dict(q=P + 8), ALIGN), (dict(cu=P + 2), ALIGN), (dict(kv_data=P + 8), ALIGN), (dict(kv_scale=P + 8), ALIGN),
    (dict(out=P + 8), ALIGN), (dict(out_f32=P + 8), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_dense(lib, change, status):
    assert call(lib.csa2_paged_attn, DENSE, DENSE_GOOD, **change) == status


def test_dense_refuses_more_tiles_than_it_counts(lib):
    """2^24 tiles a token: a CTA (of 152, the number without a device too) may have 2^30."""
    many = dict(page=1 << 20, n_pages=1, max_pages=2048, cu=P)
    for n in (9728, 12000, 1 << 20):
        assert call(lib.csa2_paged_attn, DENSE, DENSE_GOOD, **many, n=n) == SHAPE
    assert call(lib.csa2_paged_attn, DENSE, DENSE_GOOD, **many, n=9000) == WORKSPACE


def test_workspace_sizes(lib):
    sparse = lib.csa2_paged_sparse_attn_workspace_size
    assert sparse(32, 1, 512, 128) > sparse(32, 1, 256, 128) > 0
    assert sparse(0, 1, 512, 128) == sparse(1, 0, 512, 128) == sparse(1, 1, -1, 128) == 0
    dense = lib.csa2_paged_attn_workspace_size
    assert dense(1, 1) == dense(1 << 20, 7) > 0  # two parts per SM, whatever the batch
    assert dense(0, 1) == dense(1, 0) == 0


NO_POOL = dict(n_pages=0, kv_data=None, kv_scale=None)


def test_a_pool_without_pages_needs_no_planes(lib):
    keys = dict(ik_data=None, ik_scale=None)
    assert call(lib.csa2_paged_kv_append, APPEND, APPEND_GOOD, **NO_POOL, **keys, B=0) == OK
    # (beside a second thing that is wrong, so that nothing is enqueued)
    assert call(lib.csa2_paged_kv_append, APPEND, APPEND_GOOD, **NO_POOL, **keys, kv=P + 8) == ALIGN
    assert call(lib.csa2_paged_index_score, SCORE, SCORE_GOOD, n_pages=0, **keys, q=P + 8) == ALIGN
    assert call(lib.csa2_paged_sparse_attn_decode, SPARSE, SPARSE_GOOD, **NO_POOL) == WORKSPACE
    assert call(lib.csa2_paged_attn, DENSE, DENSE_GOOD, **NO_POOL) == WORKSPACE
    # one that has pages does
    for missing in ("kv_data", "kv_scale", "ik_data", "ik_scale"):
        assert call(lib.csa2_paged_kv_append, APPEND, APPEND_GOOD, **{missing: None}, n_pages=1) == ARG


def test_streams_without_the_raw_handle(monkeypatch):
    """The current stream's handle, whether or not torch gives it without a Stream object; a given stream's as it is."""
    from fp4_kv_cache_02_gb300 import csa2

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    monkeypatch.setattr(csa2.torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(csa2.torch.cuda, "current_stream", lambda: Stream(77))
    monkeypatch.setattr(csa2, "_raw_stream", lambda device: 70 + device)
    assert csa2._s(None) == 73 and csa2._s(Stream(5)) == 5
    monkeypatch.setattr(csa2, "_raw_stream", None)
    assert csa2._s(None) == 77 and csa2._s(Stream(5)) == 5
