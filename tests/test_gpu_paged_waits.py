"""What follows in the dense paged attention and in the index scans when a
device-side wait runs out.

No input makes a wait run out, so the kernels are compiled once more with short
waits: some or all CTAs of a call then give up, at different points of their
runs. The call has to end, report TIMEOUT, write nothing outside its
outputs and its workspace and leave the device as usable as before; a call in
which no wait ran out has the bits of the library's own.
"""

import concurrent.futures
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TIMEOUT = -5
LIMITS = (100, 400, 1600, 2000, 2400, 3200, 16000)  # clocks
SHORT = ("paged_attn.cu", "index_score.cu")


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    """{limit: the library with waits of that many clocks}"""
    from fp4_kv_cache_02_gb300 import _build
    _build.build()
    to = tmp_path_factory.mktemp("waits")
    rest = [os.path.join(_build.OBJ, f[:-3] + ".o") for f in sorted(os.listdir(_build.CSRC))
            if f.endswith(".cu") and f not in SHORT]

    def one(limit):
        short = f"-DCSA2_WAIT_LIMIT={limit}ull"
        obj, lib = str(to / f"{limit}_%s.o"), str(to / f"libhasty_{limit}.so")
        nvcc = _build._nvcc()
        for f in SHORT:
            subprocess.run([nvcc, *_build.ARCH, *_build.NVCC_FLAGS, short, "-c", os.path.join(_build.CSRC, f), "-o", obj % f],
                           check=True, capture_output=True)
        subprocess.run([nvcc, *_build.ARCH, "-shared", "-o", lib, *[obj % f for f in SHORT], *rest, "-lcudart_static", "-ldl",
                        "-lrt", "-lpthread"], check=True, capture_output=True)
        return ctypes.CDLL(lib)

    with concurrent.futures.ThreadPoolExecutor(len(LIMITS)) as ex:
        libs = dict(zip(LIMITS, ex.map(one, LIMITS)))
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    for lib in libs.values():
        lib.csa2_paged_attn.argtypes = [vp, i32, vp, i32, vp, vp, i64, i32, vp, i32, vp, i32, ctypes.c_float, vp, vp, vp, vp,
                                        ctypes.c_size_t, vp]
        lib.csa2_paged_index_score.argtypes = [vp, vp, vp, i32, vp, vp, i64, i32, vp, i32, vp, i64, vp, vp, vp]
        lib.csa2_index_score.argtypes = [vp, vp, vp, i32, vp, vp, i64, vp, vp, i64, vp, vp]
        lib.csa2_get_last_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    return libs


def device_status(lib, stream):
    status = ctypes.c_int(1)
    assert lib.csa2_get_last_error(stream, ctypes.byref(status)) == 0
    return status.value


class Batch:
    def __init__(self, csa2, runs, lens, page, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        places = [-(-n // page) for n in lens]
        pages = sum(places)
        order = torch.randperm(pages, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), max(places)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(places):
            self.table[b, :k] = order[at:at + k]
            at += k
        rows = torch.randn(pages * page, 512, generator=g, device="cuda").bfloat16()
        d, s = csa2.pack_kv_fp4(rows)
        self.data, self.scale = d.view(pages, page, 256), s.view(torch.uint8).view(pages, page, 32)
        self.n_visible = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.cumsum([2] + runs).tolist(), dtype=torch.int32, device="cuda")
        self.n = sum(runs) + 4
        self.q = (torch.randn(self.n, 64, 512, generator=g, device="cuda") * 512 ** -0.5).bfloat16()
        self.q[:2] = self.q[-2:] = float("nan")
        self.room = csa2.paged_attn_workspace(self.n, len(lens)).numel()
        self.space = torch.full((self.room + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        shift = -self.space.data_ptr() % 256
        self.ws = self.space[shift:shift + self.room]

    def outputs(self):
        return (torch.full_like(self.q, 7.0), torch.full(self.q.shape, 7.0, device="cuda"),
                torch.full((self.n, 64), 7.0, device="cuda"))

    def call(self, csa2):
        o = self.outputs()
        csa2.csa2_paged_attn(self.q, self.data, self.scale, self.table, self.n_visible, o[0], self.ws, cu_q=self.cu, out_f32=o[1],
                             lse=o[2])
        return o

    def hasty_call(self, lib):
        o = self.outputs()
        stream = torch.cuda.current_stream().cuda_stream
        rc = lib.csa2_paged_attn(self.q.data_ptr(), self.n, self.cu.data_ptr(), self.table.shape[0], self.data.data_ptr(),
                                 self.scale.data_ptr(), self.data.shape[0], self.data.shape[1], self.table.data_ptr(),
                                 self.table.shape[1], self.n_visible.data_ptr(), 1, 1.0, o[0].data_ptr(), o[1].data_ptr(),
                                 o[2].data_ptr(), self.ws.data_ptr(), self.room, stream)
        assert rc == 0
        return o, device_status(lib, stream)


@pytest.mark.parametrize("runs,lens,page", [
    ([1], [200], 16),
    ([1, 1], [30000, 9000], 64),                       # tokens over many CTAs
    ([3, 0, 1, 90], [300, 50, 5000, 91], 32),          # tokens of one tile and of many, a run with both
    ([400], [420], 128),                               # many tokens to a CTA
])
def test_waits_that_run_out(csa2, hasty, runs, lens, page):
    c = Batch(csa2, runs, lens, page, 5 + len(lens))
    want = c.call(csa2)
    assert csa2.csa2_get_last_error() == 0
    seen = {}
    for limit in LIMITS:
        for _ in range(4):
            got, status = c.hasty_call(hasty[limit])
            assert status in (0, TIMEOUT)
            seen.setdefault(limit, set()).add(status)
            for x, y in zip(got, want):
                assert torch.all(x[:2] == 7.0) and torch.all(x[-2:] == 7.0)
                assert status == TIMEOUT or torch.equal(x, y)
            edge = c.ws.data_ptr() - c.space.data_ptr()
            assert torch.all(c.space[:edge] == 0xA5) and torch.all(c.space[edge + c.room:] == 0xA5)
        # the next call is not touched by what was given up
        for x, y in zip(c.call(csa2), want):
            assert torch.equal(x, y)
    assert csa2.csa2_get_last_error() == 0
    assert seen[LIMITS[0]] == {TIMEOUT}, seen


@pytest.mark.parametrize("lens", [[40], [3000, 0, 700, 9000], [20000] * 12])
@pytest.mark.parametrize("form", ["flat", "paged", "claimed"])
def test_scans_whose_waits_run_out(csa2, hasty, lens, form):
    g = torch.Generator(device="cuda").manual_seed(9)
    B, page = len(lens), 64
    places = -(-max(lens) // 128) * 128 // page
    q, qs = csa2.quant_mxfp4(torch.randn(B, 32, 128, generator=g, device="cuda").bfloat16())
    k, ks = csa2.quant_mxfp4(torch.randn(B * places * page, 128, generator=g, device="cuda").bfloat16())
    w = torch.rand(B, 32, generator=g, device="cuda")
    n_visible = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.arange(B * places, dtype=torch.int32, device="cuda").view(B, places)
    n_pos = max(lens)
    counters = torch.zeros(2 * B, dtype=torch.int32, device="cuda")
    room = torch.empty(B * n_pos + 64, device="cuda")
    scores = room[32:-32].view(B, n_pos)
    stream = torch.cuda.current_stream().cuda_stream

    def call(lib):
        room.fill_(5.0)
        if form == "flat":
            rc = lib.csa2_index_score(q.data_ptr(), qs.data_ptr(), w.data_ptr(), B, k.data_ptr(), ks.data_ptr(), places * page,
                                      n_visible.data_ptr(), None, n_pos, scores.data_ptr(), stream)
        else:
            rc = lib.csa2_paged_index_score(q.data_ptr(), qs.data_ptr(), w.data_ptr(), B, k.data_ptr(), ks.data_ptr(), B * places,
                                            page, table.data_ptr(), places, n_visible.data_ptr(), n_pos, scores.data_ptr(),
                                            counters.data_ptr() if form == "claimed" else None, stream)
        assert rc == 0
        status = device_status(lib, stream)
        assert torch.all(room[:32] == 5.0) and torch.all(room[-32:] == 5.0)
        assert not counters.any()
        return scores.clone(), status

    whole = csa2.lib()
    want, status = call(whole)
    assert status == 0
    seen = {}
    for limit in LIMITS:
        for _ in range(4):
            got, status = call(hasty[limit])
            assert status in (0, TIMEOUT)
            seen.setdefault(limit, set()).add(status)
            assert status == TIMEOUT or torch.equal(got, want)
        again, status = call(whole)
        assert status == 0 and torch.equal(again, want)
    assert TIMEOUT in seen[LIMITS[0]], seen
