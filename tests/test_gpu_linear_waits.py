"""What follows in the products with 4-bit weights when a device-side wait runs out.

No input makes a wait run out, so the kernels are compiled once more with short
waits: some or all CTAs of a call then give up, at different points of their runs.
The call has to end, report TIMEOUT, write nothing outside its outputs and its
workspace and leave the device as usable as before; a call in which no wait ran out
has the bits of the library's own.
"""

import concurrent.futures
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu
TIMEOUT = -5
LIMITS = (100, 800, 1600, 2400, 3200, 6400, 20000)  # clocks


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
    rest = [os.path.join(_build.OBJ, f[:-3] + ".o") for f in sorted(os.listdir(_build.CSRC)) if f.endswith(".cu") and f != "linear.cu"]

    def one(limit):
        obj, lib = str(to / f"{limit}.o"), str(to / f"libhasty_{limit}.so")
        nvcc = _build._nvcc()
        subprocess.run([nvcc, *_build.ARCH, *_build.NVCC_FLAGS, f"-DCSA2_WAIT_LIMIT={limit}ull", "-c",
                        os.path.join(_build.CSRC, "linear.cu"), "-o", obj], check=True, capture_output=True)
        subprocess.run([nvcc, *_build.ARCH, "-shared", "-o", lib, obj, *rest, "-lcudart_static", "-ldl", "-lrt", "-lpthread"],
                       check=True, capture_output=True)
        return ctypes.CDLL(lib)

    with concurrent.futures.ThreadPoolExecutor(len(LIMITS)) as ex:
        libs = dict(zip(LIMITS, ex.map(one, LIMITS)))
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    for lib in libs.values():
        lib.csa2_fp4_linear.argtypes = [vp, i32, vp, i32, i32, i32, ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp]
        lib.csa2_get_last_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    return libs


def device_status(lib, stream):
    status = ctypes.c_int(1)
    assert lib.csa2_get_last_error(stream, ctypes.byref(status)) == 0
    return status.value


# (tokens, inputs, outputs): own terms in clusters; terms ahead in clusters, one and two CTAs to an SM; runs, whole and in
# parts; bf16 values, whole and in clusters
CASES = [(1, 8192, 600), (3, 2048, 5000), (8, 4096, 900), (12, 4096, 6000), (30, 4096, 900), (9, 1024, 12000), (32, 2816, 11000),
         (50, 4096, 9000), (90, 4096, 500), (300, 1024, 9000)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("form", ["e8m0", "e4m3"])
def test_products_whose_waits_run_out(csa2, hasty, case, form):
    run_out(csa2, hasty, case, form)


# runs over more tiles than one wave holds, two CTAs to an SM by themselves
@pytest.mark.parametrize("case", [(9, 512, 40000), (32, 1056, 20000), (50, 2816, 10000), (12, 800, 25000)])
@pytest.mark.parametrize("form", ["e8m0", "e4m3"])
def test_products_of_many_tiles_whose_waits_run_out(csa2, hasty, case, form):
    run_out(csa2, hasty, case, form)


def run_out(csa2, hasty, case, form):
    T, n_in, n_out = case
    g = torch.Generator(device="cuda").manual_seed(T)
    data = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(40, 60, (n_out, n_in // (16 if form == "e4m3" else 32)), generator=g, device="cuda", dtype=torch.uint8)
    if form == "e8m0":
        scale += 80
    w = csa2.fp4_weights(data, scale, form)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    kind = csa2.FP4_FORMATS[form]
    need = csa2.lib().csa2_fp4_linear_workspace_size(T, n_in, kind)
    room = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    shift = -room.data_ptr() % 256
    ws = room[shift:shift + need]
    big = torch.full((T * n_out + 64,), 7.0, device="cuda")
    out = big[32:32 + T * n_out].view(T, n_out)
    csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out)
    want = out.clone()
    assert csa2.csa2_get_last_error() == 0
    stream = torch.cuda.current_stream().cuda_stream
    for limit, lib in hasty.items():
        big.fill_(7.0)
        torch.cuda.synchronize()
        rc = lib.csa2_fp4_linear(x.data_ptr(), T, w.data_ptr(), n_out, n_in, kind, 1.0, None, out.data_ptr(), ws.data_ptr(), need, stream)
        assert rc == 0
        torch.cuda.synchronize()
        status = device_status(lib, stream)
        assert status == TIMEOUT if limit == LIMITS[0] else status in (0, TIMEOUT), (limit, status)
        if status == 0:
            assert torch.equal(out, want), limit
        assert (big[:32] == 7.0).all() and (big[32 + T * n_out:] == 7.0).all()
        assert (room[:shift] == 0xA5).all() and (room[shift + need:] == 0xA5).all()
        out.fill_(7.0)
        csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out)  # the device and the workspace serve the next call
        assert torch.equal(out, want) and csa2.csa2_get_last_error() == 0
