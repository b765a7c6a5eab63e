"""The first calls of a process, made by several host threads at once: what they look up
or set up once (kernels' shared memory, the driver's encoder of tensor maps) is there
for each of them."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading
import torch
from fp4_kv_cache_02_gb300 import csa2

N, T, n_in, n_out = 12, 80, 256, 300
g = torch.Generator(device="cuda").manual_seed(1)
data = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
scale = torch.randint(120, 130, (n_out, n_in // 32), generator=g, device="cuda", dtype=torch.uint8)
w = csa2.fp4_weights(data, scale, "e8m0")
x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
outs = [torch.zeros(T, n_out, device="cuda") for _ in range(N)]
spaces = [csa2.fp4_linear_workspace(T, n_in, "e8m0") for _ in range(N)]
streams = [torch.cuda.Stream() for _ in range(N)]
torch.cuda.synchronize()
meet, failed = threading.Barrier(N), []


def go(i):
    try:
        torch.cuda.set_device(0)
        meet.wait()
        csa2.csa2_fp4_linear(x, w, None, spaces[i], "e8m0", out_f32=outs[i], stream=streams[i])
    except Exception as e:
        failed.append(e)


threads = [threading.Thread(target=go, args=(i,)) for i in range(N)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not failed, failed
assert outs[0].abs().sum() > 0 and all(torch.equal(o, outs[0]) for o in outs)
assert csa2.csa2_get_last_error() == 0
print("ok")
"""


@pytest.mark.parametrize("again", range(3))
def test_first_calls_of_several_threads(again):
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-3000:]
