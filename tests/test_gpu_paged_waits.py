"""What follows in the dense paged attention when a device-side wait runs out.

No input makes a wait run out, so the kernel is compiled once more with few
tries to a wait: some or all CTAs of a call then give up, at different points of
their runs. The call has to end, report TIMEOUT, write nothing outside its
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
TRIES = (1, 4, 16, 64)


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    """{tries: the library with that many to a wait}"""
    from fp4_kv_cache_02_gb300 import _build
    _build.build()
    to = tmp_path_factory.mktemp("waits")
    rest = [os.path.join(_build.OBJ, f[:-3] + ".o") for f in sorted(os.listdir(_build.CSRC))
            if f.endswith(".cu") and f != "paged_attn.cu"]

    def one(tries):
        obj, lib = str(to / f"paged_attn_{tries}.o"), str(to / f"libhasty_{tries}.so")
        nvcc = _build._nvcc()
        subprocess.run([nvcc, *_build.ARCH, *_build.NVCC_FLAGS, f"-DCSA2_PAGED_ATTN_WAIT_TRIES={tries}u", "-c",
                        os.path.join(_build.CSRC, "paged_attn.cu"), "-o", obj], check=True, capture_output=True)
        subprocess.run([nvcc, *_build.ARCH, "-shared", "-o", lib, obj, *rest, "-lcudart_static", "-ldl", "-lrt", "-lpthread"],
                       check=True, capture_output=True)
        return ctypes.CDLL(lib)

    with concurrent.futures.ThreadPoolExecutor(len(TRIES)) as ex:
        libs = dict(zip(TRIES, ex.map(one, TRIES)))
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    for lib in libs.values():
        lib.csa2_paged_attn.argtypes = [vp, i32, vp, i32, vp, vp, i64, i32, vp, i32, vp, i32, ctypes.c_float, vp, vp, vp, vp,
                                        ctypes.c_size_t, vp]
        lib.csa2_get_last_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    return libs


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
        status = ctypes.c_int(1)
        assert lib.csa2_get_last_error(stream, ctypes.byref(status)) == 0
        return o, status.value


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
    for tries in TRIES:
        for _ in range(4):
            got, status = c.hasty_call(hasty[tries])
            assert status in (0, TIMEOUT)
            seen.setdefault(tries, set()).add(status)
            for x, y in zip(got, want):
                assert torch.all(x[:2] == 7.0) and torch.all(x[-2:] == 7.0)
                assert status == TIMEOUT or torch.equal(x, y)
            edge = c.ws.data_ptr() - c.space.data_ptr()
            assert torch.all(c.space[:edge] == 0xA5) and torch.all(c.space[edge + c.room:] == 0xA5)
        # the next call is not touched by what was given up
        for x, y in zip(c.call(csa2), want):
            assert torch.equal(x, y)
    assert csa2.csa2_get_last_error() == 0
    assert seen[1] == {TIMEOUT}, seen
