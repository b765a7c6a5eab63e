"""Products with 4-bit weights (csa2_fp4_weights, csa2_fp4_linear) against the
formula in 64 bits.

Tolerance. With A = sum_k |x_k W_k|, and M the same sum with every |x_k| replaced
by the largest of its block: the eight terms leave out at most 2^-22 M; their
magnitudes add up to at most 4 A + M 2^-20 (digits -4 .. 3 in base 8: the first one that
is not 0 is followed by at most 4/7 of its place, so the value is at least 3/7 of that
place's unit n units, the sum of all at most n + 4/7, and the rounding to the grid adds
less than a unit of the last place, 2^-20 of the largest); each tensor core product of 64
channels and the sum it is added to are taken to be off by 2^-22 of their
magnitudes (two roundings of fp32), which the ceil(n_in / 64) products of a column
add up; then nine fp32 operations join the columns and at most nine the parts and
factors. |error| <= scale * (2^-22 M + (n_in / 64 + 20) 2^-22 (4 A + 2^-20 M)). bf16 adds half a
step, 2^-9 of the value (2^-8 covers both).
"""

import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
PER = {"e8m0": 32, "e4m3": 16}


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def packed(g, n_out, n_in, form, lo=-6, hi=6):
    """Any codes, scales of 2^lo .. 2^hi (E4M3 ones with any fraction)."""
    data = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    e = torch.randint(lo, hi + 1, (n_out, n_in // PER[form]), generator=g, device="cuda")
    if form == "e8m0":
        return data, (e + 127).to(torch.uint8)
    m = torch.randint(0, 8, e.shape, generator=g, device="cuda")
    return data, ((e + 7) * 8 + m).clamp(0, 126).to(torch.uint8)


def values(data, scale, form):
    v = torch.tensor(VALUES, dtype=torch.float64, device="cuda")
    w = torch.stack([v[(data & 15).long()], v[(data >> 4).long()]], -1).flatten(-2)
    if form == "e4m3":
        s = scale.view(torch.float8_e4m3fn).double()
    else:
        s = torch.exp2(scale.double() - 127)
    return w * s.repeat_interleave(PER[form], -1)


def call(csa2, x, data, scale, form, factor=1.0, f32=True):
    w = csa2.fp4_weights(data, scale, form)
    out = torch.full((x.shape[0], data.shape[0]), 7.0, dtype=torch.bfloat16, device="cuda")
    out32 = torch.full(out.shape, 7.0, device="cuda") if f32 else None
    csa2.csa2_fp4_linear(x, w, out, csa2.fp4_linear_workspace(x.shape[0], x.shape[1], form), form, scale=factor, out_f32=out32)
    assert csa2.csa2_get_last_error() == 0
    return out, out32


def check(x, data, scale, form, out, out32, factor=1.0):
    xd, w = x.double(), values(data, scale, form)
    n_in = x.shape[1]
    ref = factor * (xd @ w.T)
    A = xd.abs() @ w.abs().T
    M = xd.abs().unflatten(-1, (-1, PER[form])).amax(-1).repeat_interleave(PER[form], -1) @ w.abs().T
    bound = abs(factor) * (2.0 ** -22 * M + (n_in / 64 + 20) * 2.0 ** -22 * (4 * A + 2.0 ** -20 * M))
    assert (out32.double() - ref).abs().le(bound).all(), ((out32.double() - ref).abs() / bound.clamp(min=1e-300)).max()
    assert torch.equal(out, out32.bfloat16())


SHAPES = [(1, 32, 1), (1, 64, 128), (2, 256, 129), (3, 288, 257), (4, 4096, 640), (5, 992, 77), (8, 1024, 300), (9, 2048, 130),
          (16, 512, 1000), (17, 800, 131), (33, 32, 70), (33, 64, 70), (49, 2336, 600), (257, 320, 200), (300, 1024, 129),
          (1021, 288, 300), (65, 64, 70), (70, 32, 129), (50, 288, 10000), (17, 512, 12000), (9, 2336, 9900), (1, 96, 40000),
          (3, 320, 39001), (16, 2048, 10000), (128, 512, 20000), (31, 96, 640), (32, 4096, 384), (33, 1056, 200), (64, 256, 513), (100, 2080, 70),
          (1, 32768, 130), (40, 8192, 1)]


@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("shape", SHAPES)
def test_against_64_bits(csa2, shape, form):
    T, n_in, n_out = shape
    g = gen(T * 7 + n_in + n_out)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    data, scale = packed(g, n_out, n_in, form)
    out, out32 = call(csa2, x, data, scale, form, 0.37)
    check(x, data, scale, form, out, out32, 0.37)


# more tiles than one wave holds: equal runs over their chunks, tiles in one part and in two (and past it: (16, 512, 38900)
# is the last that is one wave, as (17, 800, 19400) is of tiles of more tokens)
RUNS = [(17, 512, 20000), (32, 1056, 19500), (5, 96, 40000), (16, 2080, 39001), (50, 800, 10000), (64, 4128, 10100),
        (33, 32, 10000), (3000, 32, 1000), (16, 512, 38900), (17, 800, 19400), (6, 288, 25000), (12, 4096, 2048), (40, 2080, 4000)]


@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("shape", RUNS)
def test_many_tiles_against_64_bits(csa2, shape, form):
    test_against_64_bits(csa2, shape, form)


@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("shape", [(1, 64, 128), (3, 96, 70), (8, 1024, 256), (20, 4096, 200), (70, 352, 129)])
def test_whole_numbers_are_exact(csa2, shape, form):
    """Integers of eight bits times multiples of 1/2 that sum below 2^23: every term, product and sum is exact."""
    T, n_in, n_out = shape
    g = gen(5)
    x = torch.randint(-255, 256, (T, n_in), generator=g, device="cuda").bfloat16()
    data, scale = packed(g, n_out, n_in, form, 0, 1)
    if form == "e4m3":
        scale &= 0x78  # powers of two
    out, out32 = call(csa2, x, data, scale, form)
    ref = x.double() @ values(data, scale, form).T
    assert ref.abs().max() < 2 ** 23
    assert torch.equal(out32.double(), ref)
    assert torch.equal(out, out32.bfloat16())


@pytest.mark.parametrize("form", PER)
def test_channels_of_all_sizes(csa2, form):
    """One large channel to a block, the others down to 2^-30 of it: what the block's largest leaves of them."""
    T, n_in, n_out = 12, 512, 140
    g = gen(9)
    e = torch.randint(-30, 1, (T, n_in), generator=g, device="cuda").float()
    x = (torch.randn(T, n_in, generator=g, device="cuda").clamp(-3, 3) * torch.exp2(e))
    x[:, ::PER[form]] = 3.0 * torch.sign(x[:, ::PER[form]])
    x = x.bfloat16()
    data, scale = packed(g, n_out, n_in, form)
    out, out32 = call(csa2, x, data, scale, form)
    check(x, data, scale, form, out, out32)
    # the large channels' weights are zero: the others alone, each off by 2^-22 of the largest at most
    data[:, ::PER[form] // 2] &= 0xF0
    out, out32 = call(csa2, x, data, scale, form)
    check(x, data, scale, form, out, out32)
    w = values(data, scale, form)
    small = x.double().abs().le(3.0 * 2.0 ** -14)
    left = (3.0 * 2.0 ** -22 * w.abs().T[None] * small[..., None]).sum(1)
    A = x.double().abs() @ w.abs().T
    assert (out32.double() - x.double() @ w.T).abs().le(left + (n_in / 64 + 20) * 2.0 ** -20 * A).all()


@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("power", [-120, -60, 60, 110])
@pytest.mark.parametrize("T", [2, 6, 40, 90])
def test_rows_of_all_sizes(csa2, form, power, T):
    """Powers of two pass through: the row's own scale, with rows of other sizes beside it."""
    n_in, n_out = 512, 64
    g = gen(11)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    data, scale = packed(g, n_out, n_in, form, -2, 2)
    _, base = call(csa2, x, data, scale, form)
    up = x.clone()
    up[::2] = (x[::2].double() * 2.0 ** power).bfloat16()
    _, out32 = call(csa2, up, data, scale, form)
    assert torch.equal(out32[1::2], base[1::2])
    if power > -100:
        assert torch.equal(out32[::2].double(), base[::2].double() * 2.0 ** power)
    else:  # 2^-121 of each channel may be left out
        ref = up[::2].double() @ values(data, scale, form).T
        left = 2.0 ** -121 * values(data, scale, form).abs().sum(1)
        assert (out32[::2].double() - ref).abs().le(left + 2.0 ** -16 * ref.abs().max()).all()


@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("T", [68, 34, 3, 20])
def test_zero_rows_and_rows_that_are_not_finite(csa2, form, T):
    n_in, n_out = 320, 150
    g = gen(3)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    data, scale = packed(g, n_out, n_in, form)
    _, base = call(csa2, x, data, scale, form)
    bad = x.clone()
    bad[1] = 0.0
    lines = [0, T // 2 + 1, T - 1]
    bad[lines[0], 17] = float("inf")
    bad[lines[1], 0] = float("nan")
    bad[lines[2], 319] = float("-inf")
    out, out32 = call(csa2, bad, data, scale, form)
    wrong = torch.zeros(T, dtype=torch.bool, device="cuda")
    wrong[lines] = True
    assert not out32[wrong].isfinite().any() and not out[wrong].isfinite().any()
    assert (out32[1] == 0).all()
    wrong[1] = True
    assert torch.equal(out32[~wrong], base[~wrong])


@pytest.mark.parametrize("T", [2, 20, 80])
def test_extreme_scales(csa2, T):
    """E8M0 from 2^-127 to 2^120, E4M3 subnormals and 448; an E8M0 NaN spoils its own output."""
    g = gen(4)
    x = torch.randn(T, 256, generator=g, device="cuda").bfloat16()
    data, _ = packed(g, 40, 256, "e8m0")
    for code in (0, 1, 60, 247):
        scale = torch.full((40, 8), code, dtype=torch.uint8, device="cuda")
        out, out32 = call(csa2, x, data, scale, "e8m0")
        ref = x.double() @ values(data, scale, "e8m0").T
        tiny = 2.0 ** -149 * 64  # where the sums are fp32 subnormals
        A = x.double().abs() @ values(data, scale, "e8m0").abs().T
        assert (out32.double() - ref).abs().le(2.0 ** -15 * A + (tiny if code < 2 else 0)).all()
    scale[:] = 120
    _, base = call(csa2, x, data, scale, "e8m0")
    scale[7, 3] = 255
    _, out32 = call(csa2, x, data, scale, "e8m0")
    assert out32[:, 7].isnan().all()
    out32[:, 7] = base[:, 7]
    assert torch.equal(out32, base)
    scale = torch.randint(0, 127, (40, 16), generator=g, device="cuda", dtype=torch.uint8)
    out, out32 = call(csa2, x, data, scale, "e4m3")
    check(x, data, scale, "e4m3", out, out32)


@pytest.mark.parametrize("form", PER)
def test_weights_of_the_librarys_encoders(csa2, form):
    g = gen(8)
    n_out, n_in = 200, 1024
    w = torch.randn(n_out, n_in, generator=g, device="cuda").bfloat16()
    if form == "e8m0":
        data, scale = csa2.quant_mxfp4(w)
        back = torch.empty(n_out, n_in, device="cuda")
        csa2.csa2_dequant_mxfp4(data, scale, back)
    else:
        data, scale = csa2.pack_kv_fp4(w.view(-1, 512))
        back = torch.empty(n_out * n_in // 512, 512, dtype=torch.bfloat16, device="cuda")
        csa2.csa2_unpack_kv_fp4(data, scale, back)
        data, scale, back = data.view(n_out, -1), scale.view(n_out, -1), back.view(n_out, n_in)
    assert torch.equal(values(data, scale, form), back.double())
    x = torch.randn(7, n_in, generator=g, device="cuda").bfloat16()
    out, out32 = call(csa2, x, data, scale, form)
    check(x, data, scale, form, out, out32)


def test_the_layout_holds_every_code_and_scale_once(csa2):
    """Rows and inputs past the matrix are zeros, nothing else is written."""
    g = gen(2)
    for form, (n_out, n_in) in itertools.product(PER, [(1, 32), (129, 288), (128, 256)]):
        data, scale = packed(g, n_out, n_in, form)
        size = csa2.csa2_fp4_weights_size(n_out, n_in, form)
        room = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        csa2.csa2_fp4_weights(data, scale, room, form)
        assert (room[size:] == 0xA5).all()
        blocks = room[:size].view(-1, 16384 + (2048 if form == "e4m3" else 1024))
        assert blocks[:, :16384].long().sum() == data.long().sum()
        assert blocks[:, 16384:].long().sum() == scale.long().sum()


@pytest.mark.parametrize("form", PER)
def test_nothing_is_written_outside(csa2, form):
    T, n_in, n_out = 37, 544, 131
    g = gen(6)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    data, scale = packed(g, n_out, n_in, form)
    w = csa2.fp4_weights(data, scale, form)
    need = csa2.lib().csa2_fp4_linear_workspace_size(T, n_in, csa2.FP4_FORMATS[form])
    room = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = room[-room.data_ptr() % 256:][:need]
    big = torch.full((T * n_out + 64,), 7.0, device="cuda")
    out32 = big[32:32 + T * n_out].view(T, n_out)
    csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out32)
    _, want = call(csa2, x, data, scale, form)
    assert torch.equal(out32, want)
    assert (big[:32] == 7.0).all() and (big[32 + T * n_out:] == 7.0).all()
    lo = ws.data_ptr() - room.data_ptr()
    assert (room[:lo] == 0x5A).all() and (room[lo + need:] == 0x5A).all()


@pytest.mark.parametrize("form", PER)
def test_same_bits_again_on_another_stream_and_in_a_graph(csa2, form):
    T, n_in, n_out = 3, 4096, 700
    g = gen(12)
    x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
    data, scale = packed(g, n_out, n_in, form)
    w = csa2.fp4_weights(data, scale, form)
    ws = csa2.fp4_linear_workspace(T, n_in, form)
    first = torch.empty(T, n_out, device="cuda")
    csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(first)
    with torch.cuda.stream(side):
        csa2.csa2_fp4_linear(x, w, None, csa2.fp4_linear_workspace(T, n_in, form), form, out_f32=other)
    side.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(first)
    with torch.cuda.graph(graph):
        csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out)
    for i in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2.0 * first)


def test_calls_behind_one_another_share_a_workspace(csa2):
    """Sizes and formats in turn, no wait between the calls: each call's terms are read before the next writes its own."""
    g = gen(14)
    cases = []
    for form, (T, n_in, n_out) in itertools.product(PER, [(1, 4096, 640), (32, 2048, 1000), (5, 8192, 300), (70, 512, 2000)]):
        x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
        data, scale = packed(g, n_out, n_in, form)
        w = csa2.fp4_weights(data, scale, form)
        want = torch.empty(T, n_out, device="cuda")
        csa2.csa2_fp4_linear(x, w, None, csa2.fp4_linear_workspace(T, n_in, form), form, out_f32=want)
        cases.append((x, w, form, want, torch.empty_like(want)))
    ws = max((csa2.fp4_linear_workspace(x.shape[0], x.shape[1], f) for x, _, f, _, _ in cases), key=lambda t: t.numel())
    torch.cuda.synchronize()
    for _ in range(5):
        for x, w, form, want, out in cases:
            csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out)
    torch.cuda.synchronize()
    for _, _, _, want, out in cases:
        assert torch.equal(out, want)
    assert csa2.csa2_get_last_error() == 0


def test_products_on_several_streams_at_once(csa2):
    """Clusters, single CTAs, runs and values of the weights beside one another, each stream with its own workspace."""
    g = gen(16)
    cases = []
    for form, (T, n_in, n_out) in itertools.product(PER, [(1, 8192, 1500), (6, 8192, 1900), (12, 1024, 21000), (30, 1024, 20000),
                                                          (90, 4096, 1100)]):
        x = torch.randn(T, n_in, generator=g, device="cuda").bfloat16()
        data, scale = packed(g, n_out, n_in, form)
        w = csa2.fp4_weights(data, scale, form)
        want = torch.empty(T, n_out, device="cuda")
        csa2.csa2_fp4_linear(x, w, None, csa2.fp4_linear_workspace(T, n_in, form), form, out_f32=want)
        cases.append((x, w, form, want))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    runs = []
    for k, s in enumerate(streams):
        ws = [csa2.fp4_linear_workspace(x.shape[0], x.shape[1], form) for x, _, form, _ in cases]
        runs.append((s, cases[k * 3:] + cases[:k * 3], max(ws, key=lambda t: t.numel()), [[] for _ in cases]))
    torch.cuda.synchronize()
    for _ in range(8):
        for s, mine, ws, outs in runs:
            with torch.cuda.stream(s):
                for (x, w, form, want), out in zip(mine, outs):
                    out.append(torch.empty_like(want))
                    csa2.csa2_fp4_linear(x, w, None, ws, form, out_f32=out[-1])
    torch.cuda.synchronize()
    for s, mine, ws, outs in runs:
        for (x, w, form, want), out in zip(mine, outs):
            assert all(torch.equal(o, want) for o in out)
    assert csa2.csa2_get_last_error() == 0


def test_a_chain_feeds_each_product_from_the_last(csa2):
    """Outputs read by the next call at once: what a kernel of this library may start early, it does not read early."""
    g = gen(15)
    n = 512
    data, scale = packed(g, n, n, "e8m0", -4, -3)
    w = csa2.fp4_weights(data, scale, "e8m0")
    ws = csa2.fp4_linear_workspace(4, n, "e8m0")
    x = torch.randn(4, n, generator=g, device="cuda").bfloat16()
    steps = [x] + [torch.empty_like(x) for _ in range(6)]
    for a, b in zip(steps, steps[1:]):
        csa2.csa2_fp4_linear(a, w, b, ws, "e8m0", scale=0.25)
    torch.cuda.synchronize()
    for a, b in zip(steps, steps[1:]):
        again = torch.empty_like(b)
        csa2.csa2_fp4_linear(a.clone(), w, again, ws, "e8m0", scale=0.25)
        torch.cuda.synchronize()
        assert torch.equal(b, again)


def test_arguments_that_are_missing(csa2):
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    data = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(8, 2, dtype=torch.uint8, device="cuda")
    good = dict(x=x, weights=csa2.fp4_weights(data, scale, "e8m0"), out=torch.empty(2, 8, dtype=torch.bfloat16, device="cuda"),
                workspace=csa2.fp4_linear_workspace(2, 64, "e8m0"), format="e8m0")
    csa2.csa2_fp4_linear(**good)
    for name in good:
        with pytest.raises(ValueError):
            csa2.csa2_fp4_linear(**{**good, name: None})
    good = dict(data=data, scale=scale, weights=good["weights"], format="e8m0")
    csa2.csa2_fp4_weights(**good)
    for name in good:
        with pytest.raises(ValueError):
            csa2.csa2_fp4_weights(**{**good, name: None})


def test_refusals_of_the_binding(csa2):
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    data = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(8, 2, dtype=torch.uint8, device="cuda")
    w = csa2.fp4_weights(data, scale, "e8m0")
    out = torch.empty(2, 8, dtype=torch.bfloat16, device="cuda")
    ws = csa2.fp4_linear_workspace(2, 64, "e8m0")
    csa2.csa2_fp4_linear(x, w, out, ws, "e8m0")
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x[:, ::2]), dict(weights=w[:100]), dict(out=out[:1]), dict(out=None),
                dict(format="mx"), dict(workspace=ws.cpu()), dict(out_f32=torch.empty(2, 9, device="cuda"))):
        with pytest.raises(ValueError):
            csa2.csa2_fp4_linear(**{**dict(x=x, weights=w, out=out, workspace=ws, format="e8m0"), **bad})
    with pytest.raises(csa2.Csa2Error):
        csa2.csa2_fp4_linear(x, w, out, ws[:128], "e8m0")
    with pytest.raises(ValueError):
        csa2.csa2_fp4_weights(data, scale, w, "e4m3")
    with pytest.raises(ValueError):
        csa2.csa2_fp4_weights(data, scale, w[:10], "e8m0")
    with pytest.raises(csa2.Csa2Error):
        csa2.fp4_weights(torch.zeros(8, 24, dtype=torch.uint8, device="cuda"), torch.zeros(8, 1, dtype=torch.uint8, device="cuda"),
                         "e8m0")
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    csa2.csa2_fp4_linear(empty, w, torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), ws, "e8m0")
    assert csa2.csa2_get_last_error() == 0
