"""Products over many inputs: the formula in 64 bits, and a time that grows with the
inputs, not with their square.

The bound is test_gpu_linear.py's.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

PER = {"e8m0": 32, "e4m3": 16}


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def packed(g, n_out, n_in, form):
    data = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(40, 64, (n_out, n_in // PER[form]), generator=g, device="cuda", dtype=torch.uint8)
    return data, scale + 80 if form == "e8m0" else scale


def values(data, scale, form):
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    v = torch.cat([v, -v])
    w = torch.stack([v[(data & 15).long()], v[(data >> 4).long()]], -1).flatten(-2)
    s = scale.view(torch.float8_e4m3fn).double() if form == "e4m3" else torch.exp2(scale.double() - 127)
    return w * s.repeat_interleave(PER[form], -1)


def call(csa2, x, data, scale, form):
    out32 = torch.full((x.shape[0], data.shape[0]), 7.0, device="cuda")
    csa2.csa2_fp4_linear(x, csa2.fp4_weights(data, scale, form), None, csa2.fp4_linear_workspace(x.shape[0], x.shape[1], form), form,
                         out_f32=out32)
    assert csa2.csa2_get_last_error() == 0
    return out32


# on both sides of 32,768 inputs, whole CTAs of channels and part ones
@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("shape", [(2, 32768, 130), (2, 32800, 130), (9, 34816, 7), (33, 65568, 20), (64, 100000, 3), (5, 1 << 20, 2), (20, 40000, 20000)])
def test_against_64_bits(csa2, shape, form):
    T, n_in, n_out = shape
    g = gen(T + n_in)
    # channels of all sizes, tokens too; the largest of a token is in its last channels, or its first
    x = torch.randn(T, n_in, generator=g, device="cuda") * torch.exp2(torch.randint(-12, 1, (T, n_in), generator=g, device="cuda").float())
    x[::2, -3] = 100.0
    x[1::2, 2] = -100.0
    x = (x * torch.exp2(torch.arange(T, device="cuda") % 7 * 9.0 - 30)[:, None]).bfloat16()
    data, scale = packed(g, n_out, n_in, form)
    out32 = call(csa2, x, data, scale, form)
    for n0 in range(0, n_out, 2000):
        w, xd = values(data[n0:n0 + 2000], scale[n0:n0 + 2000], form), x.double()
        A = xd.abs() @ w.abs().T
        M = xd.abs().unflatten(-1, (-1, PER[form])).amax(-1).repeat_interleave(PER[form], -1) @ w.abs().T
        # (with E4M3 scales a channel may be off by 2^-39 of the token's largest)
        left = 2.0 ** -39 * xd.abs().amax(-1, keepdim=True) * w.abs().sum(1) if form == "e4m3" else 0.0
        bound = 2.0 ** -22 * M + left + (n_in / 64 + 20) * 2.0 ** -22 * (4 * A + 2.0 ** -20 * M)
        assert (out32[:, n0:n0 + 2000].double() - xd @ w.T).abs().le(bound).all()


@pytest.mark.parametrize("form", PER)
def test_long_rows_of_zeros_and_rows_that_are_not_finite(csa2, form):
    T, n_in, n_out = 8, 70016, 30
    g = gen(3)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    data, scale = packed(g, n_out, n_in, form)
    base = call(csa2, x, data, scale, form)
    bad = x.clone()
    bad[1] = 0.0
    bad[0, n_in - 1], bad[4, 40000], bad[7, 0] = float("inf"), float("nan"), -float("inf")
    out = call(csa2, bad, data, scale, form)
    assert not out[[0, 4, 7]].isfinite().any() and (out[1] == 0).all()
    assert torch.equal(out[[2, 3, 5, 6]], base[[2, 3, 5, 6]])


def test_long_rows_in_a_graph_behind_one_another(csa2):
    """Terms behind their factors, and the next call's factors behind the product that reads these, in one workspace."""
    T, n_in, n_out = 6, 50016, 200
    g = gen(5)
    data, scale = packed(g, n_out, n_in, "e4m3")
    w, ws = csa2.fp4_weights(data, scale, "e4m3"), csa2.fp4_linear_workspace(T, n_in, "e4m3")
    xs = [(torch.randn(T, n_in, generator=g, device="cuda") * 2.0 ** (20 * i - 40)).bfloat16() for i in range(5)]
    want = [call(csa2, x, data, scale, "e4m3") for x in xs]
    outs = [torch.zeros_like(o) for o in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, o in zip(xs, outs):
            csa2.csa2_fp4_linear(x, w, None, ws, "e4m3", out_f32=o)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
    assert csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("form", PER)
def test_the_time_grows_with_the_inputs(csa2, form):
    """Four times the inputs: four times the work. Eight times the time is allowed; a square would be sixteen."""
    took = []
    for n_in in (1 << 21, 1 << 23):
        x = torch.ones(4, n_in, dtype=torch.bfloat16, device="cuda")
        w = torch.zeros(csa2.csa2_fp4_weights_size(1, n_in, form), dtype=torch.uint8, device="cuda")
        ws, out = csa2.fp4_linear_workspace(4, n_in, form), torch.empty(4, 1, dtype=torch.bfloat16, device="cuda")
        times = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            csa2.csa2_fp4_linear(x, w, out, ws, form)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took.append(sorted(times)[3])
    assert took[1] < 8 * took[0], took
