"""GPU parity of the paged cache: append with the position rotation, rotation of
queries and outputs, index scores, sparse and dense attention over pages.

Every reference is a plain computation in 64 bits (the packed bytes: the oracle
on values rotated in 64 bits). Tolerances, with u = 2^-11 for one rounding to
fp16 and 2^-8 for one to bf16:
  - packed bytes, counts: exact;
  - csa2_rope: one rounding to bf16 of a value within 2^-24 of the exact one;
  - scores: 32 terms summed in fp32 after exact products of blocks;
  - attention: each weight is rounded to fp16 once, and the scores carry the
    error d = 512 2^-24 max sum|q||row| of a 512-term fp32 sum, so that
    |out - ref| <= (u + 3 d + 2^-18) sum_j p_j |row_j| channel by channel (a
    weight moves by e^(2 d) at most, numerator and denominator; 2^-18 for the
    exponential, the fp32 sums and the division), and lse moves by d + 2^-18.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEVICE_ERROR = -7


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


@pytest.fixture(autouse=True)
def clean(csa2):
    csa2.csa2_get_last_error()
    yield


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(runs, first=0):
    return ints(np.cumsum([first] + list(runs)).tolist())


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def angles(n, dim, base=10000.0):
    a = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.stack([a.cos(), a.sin()], -1).float().cuda().contiguous()


def rotated(x, rope, positions, interleaved, inverse=False):
    """x [n, ..., d] in 64 bits with its last channels turned (numpy-free, on the device)."""
    dim = 2 * rope.shape[1]
    r = rope.double()[positions.long()]
    c, s = r[..., 0], r[..., 1] * (-1 if inverse else 1)
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (dim // 2,)
    c, s = c.view(shape), s.view(shape)
    y = x.double().clone()
    z = y[..., -dim:]
    u, v = (z[..., 0::2].clone(), z[..., 1::2].clone()) if interleaved else (z[..., :dim // 2].clone(), z[..., dim // 2:].clone())
    a, b = u * c - v * s, u * s + v * c
    if interleaved:
        z[..., 0::2], z[..., 1::2] = a, b
    else:
        z[..., :dim // 2], z[..., dim // 2:] = a, b
    return y


def tables(lens, page, g, extra=2, most=None, unused=-1):
    """A shuffled page table for sequences of `lens` entries, and the pool's pages."""
    need = [-(-n // page) for n in lens]
    most = max(max(need), 1) if most is None else most
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g, device="cuda").int()
    t = torch.full((len(lens), most), unused, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = order[at:at + k]
        at += k
    return t, pages


def rows_of(table, b, n, page):
    e = torch.arange(n, device="cuda")
    return table[b].long()[e // page] * page + e % page


class Cache:
    """Packed random latents and keys of `lens` entries in pages; every other byte of the pool is random."""

    def __init__(self, csa2, lens, page, seed, most=None, scale=1.0, unused=-1):
        g = gen(seed)
        self.lens, self.page = lens, page
        self.table, self.pages = tables(lens, page, g, most=most, unused=unused)
        self.n_visible = ints(lens)
        self.planes = [torch.randint(0, 256, (self.pages, page, w), generator=g, device="cuda", dtype=torch.uint8)
                       for w in (256, 32, 64, 4)]
        self.kv_data, self.kv_scale, self.ik_data, self.ik_scale = self.planes
        self.kv_scale |= 0x7F  # NaN scales wherever no entry is
        self.rows, self.flat = [], []
        for b, n in enumerate(lens):
            x, k = normal(g, n, 512, scale=scale), normal(g, n, 128)
            if n:
                packed = (*csa2.pack_kv_fp4(x), *csa2.quant_mxfp4(k))
                at = rows_of(self.table, b, n, page)
                for plane, new in zip(self.planes, packed):
                    plane.view(-1, plane.shape[-1])[at] = new
            self.rows.append(at if n else None)

    def latents(self, csa2, b):
        n = self.lens[b]
        out = torch.empty(n, 512, dtype=torch.bfloat16, device="cuda")
        if n:
            d = self.kv_data.view(-1, 256)[self.rows[b]].contiguous()
            s = self.kv_scale.view(-1, 32)[self.rows[b]].contiguous()
            csa2.csa2_unpack_kv_fp4(d, s, out)
        return out.double()

    def flat_planes(self, cap=None):
        """The same entries in the flat [B, cap, w] planes."""
        cap = cap or -(-max(max(self.lens), 1) // 128) * 128
        out = []
        for plane in self.planes:
            f = torch.zeros(len(self.lens), cap, plane.shape[-1], dtype=torch.uint8, device="cuda")
            for b, n in enumerate(self.lens):
                if n:
                    f[b, :n] = plane.view(-1, plane.shape[-1])[self.rows[b]]
            out.append(f)
        return out


# ---- the latents' encoder --------------------------------------------------------


def test_latent_codes_are_those_of_the_rounded_quotient(csa2):
    """Codes and scales of blocks of every size of bf16, signed zeros and subnormals among them, against the quotients rounded
    to fp32: the encoder divides by a corrected reciprocal."""
    g = gen(3)
    n = 1 << 14
    bits = torch.randint(0, 1 << 16, (n, 512), generator=g, device="cuda", dtype=torch.int32)
    # the blocks' values within a few octaves below a top that goes through all exponents
    top = torch.randint(0, 0x7F80, (n, 32, 1), generator=g, device="cuda", dtype=torch.int32)
    less = torch.randint(0, 4 << 7, (n, 32, 16), generator=g, device="cuda", dtype=torch.int32)
    near = (bits.view(n, 32, 16) & 0x8000) | (top - less).clamp(min=0)
    x = torch.where(torch.arange(n, device="cuda")[:, None, None] % 8 == 0, bits.view(n, 32, 16), near)
    x = torch.where((x & 0x7F80) == 0x7F80, x & 0x8000, x)  # finite
    v = (x << 16).view(torch.float32).view(n, 32, 16)
    data, scale = csa2.pack_kv_fp4(v.view(n, 512).bfloat16())
    amax = v.abs().amax(-1)
    want = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    assert torch.equal(scale.view(torch.uint8).view(n, 32), want.view(torch.uint8))
    s = want.float()[..., None]
    quotient = v / torch.where(s > 0, s, torch.ones_like(s))
    a = quotient.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int()
            + (a > 5.0).int() + 8 * torch.signbit(quotient).int())
    code = torch.where(s > 0, code, torch.zeros_like(code)).view(n, 256, 2)
    assert torch.equal(data.view(n, 256).int(), code[..., 0] + 16 * code[..., 1])


def test_latent_codes_beside_infinities_and_nans(csa2):
    """An infinity takes its block's scale to the largest and saturates; a NaN leaves its neighbours as they are."""
    x = normal(gen(4), 3, 512)
    plain, plain_scale = csa2.pack_kv_fp4(x)
    y = x.clone()
    y[0, 5], y[1, 37] = float("inf"), -float("inf")
    y[2, 100] = float("nan")
    data, scale = csa2.pack_kv_fp4(y)
    codes = torch.stack([data & 15, data >> 4], -1).view(3, 512)
    before = torch.stack([plain & 15, plain >> 4], -1).view(3, 512)
    assert int(scale[0, 0]) == int(scale[1, 2]) == 0x7E
    assert int(codes[0, 5]) == 7 and int(codes[1, 37]) == 15
    rest = torch.ones(3, 512, dtype=torch.bool, device="cuda")
    rest[0, :16], rest[1, 32:48], rest[2, 96:112] = False, False, False
    assert torch.equal(codes[rest], before[rest])
    z = x.clone()
    z[2, 100] = 0.0
    other, other_scale = csa2.pack_kv_fp4(z)
    other = torch.stack([other & 15, other >> 4], -1).view(3, 512)
    assert torch.equal(scale[2], other_scale[2])
    kept = torch.arange(512, device="cuda") != 100
    assert torch.equal(codes[2][kept], other[2][kept])


# ---- append ----------------------------------------------------------------------


def append_reference(kv, ik, runs, first, past, table, page, planes, rope, positions, interleaved):
    ref = [p.clone() for p in planes]
    at = first
    for b, T in enumerate(runs):
        if T:
            x, k = kv[at:at + T].double(), ik[at:at + T].double()
            if rope is not None:
                e = torch.arange(past[b], past[b] + T, device="cuda") if positions is None else positions[at:at + T]
                x, k = rotated(x, rope, e, interleaved), rotated(k, rope, e, interleaved)
            x, k = x.float().cpu().numpy(), k.float().cpu().numpy()
            packed = (*oracle.pack_kv_fp4(x), *oracle.quant_mxfp4(k))
            rows = rows_of(table, b, past[b] + T, page)[past[b]:]
            for plane, new in zip(ref, packed):
                plane.view(-1, plane.shape[-1])[rows] = torch.from_numpy(np.ascontiguousarray(new)).cuda()
        at += T
    return ref


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("rope_dim,interleaved", [(0, False), (32, True), (64, True), (64, False), (128, True), (128, False)])
def test_append_writes_the_oracle_s_bytes(csa2, page, rope_dim, interleaved):
    g = gen(page + rope_dim)
    runs, past = [0, 1, 37, 5, 130, 0, 1], [3, 0, 15, 250, 1, 0, 63]
    table, pages = tables([a + t for a, t in zip(past, runs)], page, g)
    n, first, behind = sum(runs), 2, 3
    kv, ik = normal(g, first + n + behind, 512, scale=3.0), normal(g, first + n + behind, 128, scale=3.0)
    kv[first::7, :32] = 0          # zero blocks, saturating and tiny magnitudes
    kv[first + 1::11, 16:48] *= 1e4
    kv[first + 2::5, 448:] *= 1e-20
    ik[first + 1::3, 64:96] = 0
    kv[:first] = kv[first + n:] = float("nan")  # rows of no sequence
    rope = angles(600, rope_dim) if rope_dim else None
    planes = [torch.randint(0, 256, (pages, page, w), generator=g, device="cuda", dtype=torch.uint8) for w in (256, 32, 64, 4)]
    ref = append_reference(kv, ik, runs, first, past, table, page, planes, rope, None, interleaved)
    out = torch.full((7,), -5, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_kv_append(kv, ik, *planes, table, ints(past), out, cu_tokens=starts(runs, first), rope=rope,
                              interleaved=interleaved)
    assert csa2.csa2_get_last_error() == 0
    for got, want in zip(planes, ref):
        assert torch.equal(got, want)
    assert out.tolist() == [a + t for a, t in zip(past, runs)]


@pytest.mark.parametrize("mode", ["separate", "inplace", "none"])
@pytest.mark.parametrize("T", [1, 3])
def test_append_of_equal_runs_equals_the_flat_append(csa2, mode, T):
    """Without a rotation the bytes are csa2_kv_append's (the pool's pages in order are flat planes)."""
    g = gen(5 + T)
    B, page, most = 33, 32, 4
    kv, ik = normal(g, B * T, 512, scale=4.0), normal(g, B * T, 128)
    past = torch.randint(0, most * page - T, (B,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.arange(B * most, dtype=torch.int32, device="cuda").view(B, most)
    flat = [torch.zeros(B, most * page, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    paged = [f.clone().view(B * most, page, -1) for f in flat]
    n1, n2 = past.clone(), past.clone()
    def into(n):
        return None if mode == "none" else n if mode == "inplace" else torch.empty_like(n)
    o1, o2 = into(n1), into(n2)
    csa2.csa2_kv_append(kv.view(B, T, 512), ik.view(B, T, 128), *flat, n1, n_visible_out=o1)
    csa2.csa2_paged_kv_append(kv, ik, *paged, table, n2, o2)
    for a, b in zip(flat, paged):
        assert torch.equal(a.view(-1), b.view(-1))
    if o1 is not None:
        assert torch.equal(o1, o2) and torch.equal(o1, past + T)
    assert csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("tokens", [1, 200])  # one and several tokens to a warp are told apart by the whole call's tokens
def test_append_of_nans_and_infinities_equals_the_flat_append(csa2, tokens):
    """Without a rotation the bytes are csa2_kv_append's for any inputs, and those of the encoders."""
    g = gen(97)
    B = 32
    kv, ik = normal(g, B * tokens, 512), normal(g, B * tokens, 128)
    for x, block in ((kv, 16), (ik, 32)):
        blocks = x.view(-1, block)
        for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
            rows = torch.arange(i, blocks.shape[0], 7, device="cuda")
            blocks[rows, torch.randint(0, block, rows.shape, generator=g, device="cuda")] = v
        blocks[5::11] = float("nan")
        blocks[6::13] *= 0
        bits = torch.randint(0, 1 << 16, blocks[8::17].shape, generator=g, device="cuda", dtype=torch.int32)
        blocks[8::17] = (bits - (1 << 15)).short().view(torch.bfloat16)
    page = 256
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    flat = [torch.zeros(B, page, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    paged = [f.clone() for f in flat]
    csa2.csa2_kv_append(kv.view(B, tokens, 512), ik.view(B, tokens, 128), *flat, ints([3] * B))
    csa2.csa2_paged_kv_append(kv, ik, *paged, table, ints([3] * B))
    assert csa2.csa2_get_last_error() == 0
    want = *csa2.pack_kv_fp4(kv), *csa2.quant_mxfp4(ik)
    for a, b, c in zip(flat, paged, want):
        assert torch.equal(a, b)
        assert torch.equal(b[:, 3:3 + tokens].reshape(B * tokens, -1), c.view(torch.uint8).view(B * tokens, -1))


def test_append_codes_of_fp32_values_beside_every_border(csa2):
    """Turned values are fp32: the encoder's codes for values within three steps of every border of every scale, and scales for
    blocks whose largest is within three steps of every border between scales, against the rounded quotients. A table of
    (c, 0) makes any fp32 value c of a row of ones."""
    def beside(x):
        bits = np.float32(x).view(np.int32)
        return [(bits + i).astype(np.int32).view(np.float32) for i in range(-3, 4)]

    scales = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    borders = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
    blocks = []
    for s in scales[1:]:
        near = [v for b in borders for v in beside(b * s)] + [s * 6] * 11
        blocks += [[6 * s] + near[15 * i:15 * i + 15] for i in range(4)]
    rng = np.random.default_rng(7)
    for lo, hi in zip(scales, scales[1:]):
        blocks += [[v] + list(v * rng.random(15, dtype=np.float32)) for v in beside(3 * (lo + hi))]
    blocks += [[v] + list(v * rng.random(15, dtype=np.float32)) for v in beside(6 * 464.0) + beside(6 * 448.0) + beside(1e30)]
    blocks += [[0.0] * 16] * (-len(blocks) % 4)
    c = torch.from_numpy(np.array(blocks, dtype=np.float32)).view(-1, 64)
    n = c.shape[0]
    rope = torch.stack([c, torch.zeros_like(c)], -1).cuda().contiguous()
    kv = torch.ones(n, 512, dtype=torch.bfloat16, device="cuda")
    kv[:, 448:] = -1.0  # the second of each pair: -c
    ik = torch.zeros(n, 128, dtype=torch.bfloat16, device="cuda")
    pages = -(-n // 16)
    planes = [torch.zeros(pages, 16, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    csa2.csa2_paged_kv_append(kv, ik, *planes, torch.arange(pages, dtype=torch.int32, device="cuda")[None], ints([0]), rope=rope)
    assert csa2.csa2_get_last_error() == 0
    v = c.view(n, 4, 16)
    want = (v.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = want.float()[..., None]
    a = v / torch.where(s > 0, s, torch.ones_like(s))
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int()
            + (a > 5.0).int())
    code = torch.where(s > 0, code, torch.zeros_like(code)).view(n, 64)
    got = torch.stack([planes[0] & 15, planes[0] >> 4], -1).view(-1, 512)[:n].int().cpu()
    scale = planes[1].view(-1, 32)[:n].cpu()
    for half, sign in ((0, 0), (1, 8)):
        assert torch.equal(scale[:, 24 + 4 * half:28 + 4 * half], want.view(torch.uint8))
        part = got[:, 384 + 64 * half:448 + 64 * half]
        negative = torch.where(s.expand(n, 4, 16).reshape(n, 64) > 0, sign, 0)
        # (a zero of either sign: the code's sign is not looked at)
        assert torch.equal(part & 7, code)
        assert torch.equal((part & 8)[code > 0], negative[code > 0].int())


def test_append_at_given_positions(csa2):
    g = gen(11)
    runs, past, page = [4, 9], [30, 2], 16
    table, pages = tables([34, 11], page, g)
    kv, ik = normal(g, 13, 512), normal(g, 13, 128)
    positions = torch.randint(0, 1 << 17, (13,), generator=g, device="cuda", dtype=torch.int32)
    rope = angles(1 << 17, 64)
    planes = [torch.zeros(pages, page, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    ref = append_reference(kv, ik, runs, 0, past, table, page, planes, rope, positions, True)
    csa2.csa2_paged_kv_append(kv, ik, *planes, table, ints(past), cu_tokens=starts(runs), rope=rope, positions=positions,
                              interleaved=True)
    for got, want in zip(planes, ref):
        assert torch.equal(got, want)


@pytest.mark.parametrize("mode", ["separate", "inplace"])
def test_append_passes_over_what_does_not_fit(csa2, mode):
    """A full sequence, a negative count and a run outside the rows change nothing; a page outside the pool and a position
    outside the table lose their entries only. All are reported."""
    g = gen(12)
    page, most = 16, 3
    past = [40, -2, 20, 0, 5]
    cu = ints([0, 10, 12, 30, 30, 34])       # runs 10 (of 8 left), 2, 18, 0, 4
    table = torch.arange(15, dtype=torch.int32, device="cuda").view(5, most)
    table[2, 2] = 99                          # sequence 2: entries 32 .. 37
    kv, ik = normal(g, 34, 512), normal(g, 34, 128)
    rope = angles(64, 32)
    positions = torch.full((34,), 7, dtype=torch.int32, device="cuda")
    positions[31] = 64                        # sequence 4's second token
    positions[33] = -1
    planes = [torch.full((15, page, w), 0xA5, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    want = [p.clone() for p in planes]
    for b, lo, n in ((2, 12, 12), (4, 30, 1), (4, 32, 1)):  # (sequence, first row, entries kept)
        e0 = past[b] + (lo - cu.tolist()[b])
        x = rotated(kv[lo:lo + n], rope, positions[lo:lo + n], False).float().cpu().numpy()
        k = rotated(ik[lo:lo + n], rope, positions[lo:lo + n], False).float().cpu().numpy()
        rows = rows_of(table, b, e0 + n, page)[e0:]
        for plane, new in zip(want, (*oracle.pack_kv_fp4(x), *oracle.quant_mxfp4(k))):
            plane.view(-1, plane.shape[-1])[rows] = torch.from_numpy(np.ascontiguousarray(new)).cuda()
    nv = ints(past)
    out = nv if mode == "inplace" else torch.empty_like(nv)
    csa2.csa2_paged_kv_append(kv, ik, *planes, table, nv, out, cu_tokens=cu, rope=rope, positions=positions)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    assert out.tolist() == [40, -2, 38, 0, 9]
    for got, ref in zip(planes, want):
        assert torch.equal(got, ref)
    # runs that are not within the rows
    nv = ints([0, 0])
    out = torch.empty_like(nv)
    before = [p.clone() for p in planes]
    csa2.csa2_paged_kv_append(kv, ik, *planes, table[:2], nv, out, cu_tokens=ints([-3, 35, 20]))
    assert csa2.csa2_get_last_error() == DEVICE_ERROR and out.tolist() == [0, 0]
    assert all(torch.equal(a, b) for a, b in zip(planes, before))


@pytest.mark.parametrize("rope_dim,interleaved", [(0, False), (64, True), (96, False), (128, True)])
def test_append_of_many_tokens_equals_the_sequences_alone(csa2, rope_dim, interleaved):
    """A call with several tokens to a warp writes what one call per sequence writes; rows of no sequence are not read."""
    g = gen(13 + rope_dim)
    runs = [30 + (97 * i * i + 5) % 301 for i in range(40)]
    runs[3] = runs[20] = 0
    runs[21] = 1
    first, n = 3, sum(runs)
    assert n > 5000
    past = [(29 * i) % 70 for i in range(40)]
    page = 32
    table, pages = tables([a + t for a, t in zip(past, runs)], page, g)
    kv, ik = normal(g, first + n + 6, 512), normal(g, first + n + 6, 128)
    kv[:first] = kv[first + n:] = float("nan")
    rope = angles(500, rope_dim) if rope_dim else None
    kept = [torch.randint(0, 256, (pages, page, w), generator=g, device="cuda", dtype=torch.uint8) for w in (256, 32, 64, 4)]
    together, alone = [p.clone() for p in kept], [p.clone() for p in kept]
    out = torch.empty(40, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_kv_append(kv, ik, *together, table, ints(past), out, cu_tokens=starts(runs, first), rope=rope,
                              interleaved=interleaved)
    at = first
    for b, t in enumerate(runs):
        csa2.csa2_paged_kv_append(kv[at:at + t], ik[at:at + t], *alone, table[b:b + 1], ints(past[b:b + 1]), rope=rope,
                                  interleaved=interleaved)
        at += t
    assert csa2.csa2_get_last_error() == 0
    assert out.tolist() == [a + t for a, t in zip(past, runs)]
    for a, b in zip(together, alone):
        assert torch.equal(a, b)


def test_append_of_nothing(csa2):
    planes = [torch.zeros(2, 16, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    kv, ik = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_kv_append(kv, ik, *planes, ints([[0], [1]]), ints([4, 9]), out)
    assert out.tolist() == [4, 9] and csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("n", [23, 6000])  # one and several tokens to a warp
@pytest.mark.parametrize("cu", [[0, 0, 0], [7, 7, 7], [23, 23, 23], [5, 6, 6], [6, 6, 9], [0, 1, 2], [21, 22, 23], [9, 4, 4],
                                [-4, -2, 0], [24, 40, 7000], [5, 2, 8]])
def test_append_of_few_rows_among_many(csa2, cu, n):
    """Rows of no sequence, and runs that are not within the rows, at every place within a warp's tokens."""
    kv, ik = normal(gen(98), n, 512), normal(gen(98), n, 128)
    planes = [torch.zeros(2, 16, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    want = [p.clone() for p in planes]
    packed = *csa2.pack_kv_fp4(kv), *csa2.quant_mxfp4(ik)
    counts = []
    for b in range(2):
        lo, hi = cu[b], cu[b + 1]
        ok = 0 <= lo <= hi <= n
        run = hi - lo if ok and hi - lo <= 13 else 0
        counts.append(3 + run)
        if run and cu == sorted(cu):
            for plane, new in zip(want, packed):
                plane[b, 3:3 + run] = new.view(torch.uint8).view(n, -1)[lo:hi]
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_kv_append(kv, ik, *planes, ints([[0], [1]]), ints([3, 3]), out, cu_tokens=ints(cu))
    refused = any(not 0 <= cu[b] <= cu[b + 1] <= n or cu[b + 1] - cu[b] > 13 for b in range(2))
    assert csa2.csa2_get_last_error() == (DEVICE_ERROR if refused else 0)
    assert out.tolist() == counts
    if cu == sorted(cu):
        for got, ref in zip(planes, want):
            assert torch.equal(got, ref)


def test_append_refuses_an_empty_angle_table(csa2):
    """A table without positions is not a missing one: nothing is written unrotated. Without tokens there is nothing to turn."""
    planes = [torch.zeros(2, 16, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    kv, ik = normal(gen(96), 2, 512), normal(gen(96), 2, 128)
    none = torch.empty(0, 32, 2, device="cuda")
    out = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="no position"):
        csa2.csa2_paged_kv_append(kv, ik, *planes, ints([[0], [1]]), ints([4, 9]), out, rope=none)
    assert out.tolist() == [-5, -5] and not any(p.any() for p in planes)
    with pytest.raises(csa2.Csa2Error):
        csa2.csa2_rope(kv[:, None], none, None, kv[:, None])
    csa2.csa2_paged_kv_append(kv[:0], ik[:0], *planes, ints([[0], [1]]), ints([4, 9]), out, rope=none)
    assert out.tolist() == [4, 9] and csa2.csa2_get_last_error() == 0


# ---- rotation ----------------------------------------------------------------------


@pytest.mark.parametrize("heads,dim,rope_dim", [(64, 512, 64), (32, 128, 64), (1, 512, 128), (3, 40, 32), (5, 32, 32)])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_rope(csa2, heads, dim, rope_dim, interleaved, inverse, inplace):
    g = gen(dim + heads)
    n, far = 37, 1 << 20
    x = normal(g, n, heads, dim)
    rope = angles(far, rope_dim)
    positions = torch.randint(0, far, (n,), generator=g, device="cuda", dtype=torch.int32)
    positions[0], positions[1] = 0, far - 1
    ref = rotated(x, rope, positions, interleaved, inverse)
    keep = x.clone()
    out = x if inplace else torch.empty_like(x)
    csa2.csa2_rope(x, rope, positions, out, interleaved=interleaved, inverse=inverse)
    assert csa2.csa2_get_last_error() == 0
    assert torch.equal(out[..., :dim - rope_dim], keep[..., :dim - rope_dim])
    err = (out.double() - ref).abs()
    assert torch.all(err <= ref.abs() * 2.0 ** -8 * (1 + 2.0 ** -14) + 1e-38)
    if not inplace:
        assert torch.equal(x, keep)


def test_rope_rows_without_positions_or_with_bad_ones(csa2):
    g = gen(3)
    x, rope = normal(g, 20, 4, 64), angles(20, 32)
    out = torch.empty_like(x)
    csa2.csa2_rope(x, rope, None, out)
    ref = rotated(x, rope, torch.arange(20, device="cuda"), False)
    assert torch.all((out.double() - ref).abs() <= ref.abs() * 2.0 ** -8 * (1 + 2.0 ** -14) + 1e-38)
    assert csa2.csa2_get_last_error() == 0
    out.fill_(9.0)
    positions = torch.arange(20, dtype=torch.int32, device="cuda")
    positions[4], positions[7] = 20, -1
    csa2.csa2_rope(x, rope, positions, out)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    assert torch.all(out[4] == 9.0) and torch.all(out[7] == 9.0)
    good = [i for i in range(20) if i not in (4, 7)]
    assert torch.all((out.double() - ref).abs()[good] <= ref.abs()[good] * 2.0 ** -8 * (1 + 2.0 ** -14) + 1e-38)


def overflowing(n, heads, dim, rope_dim):
    """(x, rope, positions): rows with infinities among the turned channels, beside finite values and beside each other, and
    with finite pairs whose turned values pass fp32's range."""
    x = normal(gen(95), n, heads, dim)
    top = float(torch.finfo(torch.bfloat16).max)
    special = [float("inf"), -float("inf"), top, -top]
    t = x[..., -rope_dim:]
    for i in range(n):
        t[i, :, i % rope_dim] = special[i % 4]
        t[i, :, (i + rope_dim // 2) % rope_dim] = special[(i // 4) % 4]
        t[i, :, (i + 1) % rope_dim] = special[(i // 16) % 4]
    rope = angles(n, rope_dim)
    return x, rope, torch.arange(n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_of_infinities_and_of_what_overflows(csa2, interleaved):
    """An infinite channel, or a pair whose turned value passes fp32's range, gives the infinities of the formula (NaN only
    where that is a difference of infinities), and other pairs are not touched by it."""
    x, rope, positions = overflowing(64, 3, 512, 64)
    out = torch.empty_like(x)
    csa2.csa2_rope(x, rope, positions, out, interleaved=interleaved)
    assert csa2.csa2_get_last_error() == 0
    # (in 64 bits a finite pair stays finite: what rounds past fp32's largest is infinite)
    ref = rotated(x, rope, positions, interleaved).float()
    assert int(torch.isinf(ref).sum()) > 400 and int(torch.isnan(ref).sum()) > 20
    assert int((torch.isinf(ref) & torch.isfinite(rotated(x, rope, positions, interleaved))).sum()) > 20
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    far = torch.isinf(ref) | torch.isnan(ref)
    assert torch.equal(out[torch.isinf(ref)].float(), ref[torch.isinf(ref)])
    # (a value within fp32's range may round past bf16's: the infinity that one rounding to bf16 gives)
    near = ref.bfloat16()
    over = torch.isinf(near) & ~far
    assert torch.equal(out[over], near[over])
    rest = ~far & ~over
    assert torch.all((out.double() - ref.double()).abs()[rest] <= ref.double().abs()[rest] * 2.0 ** -8 * (1 + 2.0 ** -14) + 1e-38)


@pytest.mark.parametrize("interleaved", [True, False])
def test_append_of_infinities_and_of_what_overflows(csa2, interleaved):
    """The same through the append: a block with an infinity has the largest scale, the infinity's code is the largest of its
    sign, and so for the keys."""
    kv, rope, positions = overflowing(64, 1, 512, 64)
    ik, _, _ = overflowing(64, 1, 128, 64)
    kv, ik = kv[:, 0].contiguous(), ik[:, 0].contiguous()
    planes = [torch.zeros(4, 16, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    csa2.csa2_paged_kv_append(kv, ik, *planes, table, ints([0]), rope=rope, interleaved=interleaved)
    assert csa2.csa2_get_last_error() == 0
    for x, data, scale, block, largest in ((kv, planes[0], planes[1], 16, 0x7E), (ik, planes[2], planes[3], 32, 253)):
        y = rotated(x, rope, positions, interleaved).float()
        codes = torch.stack([data & 15, data >> 4], -1).view(64, -1)
        infinite = torch.isinf(y)
        assert int(infinite.sum()) > 50
        assert torch.equal(codes[infinite], torch.where(y[infinite] > 0, 7, 15).to(torch.uint8))
        blocks = infinite.view(64, -1, block).any(-1)
        assert torch.all(scale.view(64, -1)[blocks] == largest)


@pytest.mark.parametrize("between", [False, True])
def test_attention_right_behind_the_rotation(csa2, between):
    """The selected attention loads its queries before it waits for the kernel before it: a rotation that is still writing them
    may not let it start, nor the attention call behind another one."""
    g = gen(104)
    n = 4096                                            # (the rotation takes 80 us, the queries are its last rows)
    c = Cache(csa2, [300], 64, 105)
    flat = c.flat_planes()
    x = normal(g, n, 64, 512, scale=512 ** -0.5)
    rope = angles(n, 64)
    idx = torch.arange(128, dtype=torch.int32, device="cuda")[None]
    swa = csa2.pack_fp8(normal(g, 1, 4, 16, 512))
    other, o3 = x[:4].view(1, 4, 64, 512).contiguous(), torch.empty(1, 4, 64, 512, dtype=torch.bfloat16, device="cuda")
    ws = [csa2.paged_sparse_attn_workspace(1, 4, 128, 16) for _ in range(3)]
    want = None
    for i in range(6):
        for call in ("paged", "flat"):
            turned = torch.zeros_like(x)
            q = turned[-4:].view(1, 4, 64, 512)
            got = torch.empty_like(q)
            torch.cuda.synchronize()
            csa2.csa2_rope(x, rope, None, turned, interleaved=True)
            if want is None:
                torch.cuda.synchronize()
            elif between:
                csa2.csa2_paged_sparse_attn_decode(other, c.kv_data, c.kv_scale, c.table, c.n_visible, idx, swa, o3, ws[0])
            if call == "paged":
                csa2.csa2_paged_sparse_attn_decode(q, c.kv_data, c.kv_scale, c.table, c.n_visible, idx, swa, got, ws[1])
            else:
                csa2.csa2_sparse_attn_decode(q, flat[0], flat[1], c.n_visible, idx, swa, got, ws[2])
            if want is None:
                want = got
            assert torch.equal(got, want), (i, call)
    assert csa2.csa2_get_last_error() == 0


# ---- index scores ---------------------------------------------------------------------


def queries(csa2, g, B):
    q, s = csa2.quant_mxfp4(normal(g, B, 32, 128))
    return q, s, torch.rand(B, 32, generator=g, device="cuda")


@pytest.mark.parametrize("page", [16, 32, 64, 128, 512])
@pytest.mark.parametrize("claimed", [False, True])
def test_scores_equal_the_flat_scan(csa2, page, claimed):
    lens = [0, 1, 127, 128, 129, 2500, 777]
    c = Cache(csa2, lens, page, 20 + page, unused=1 << 30)
    q, s, w = queries(csa2, gen(21), len(lens))
    n_pos = 2500
    flat = c.flat_planes()
    want = torch.empty(len(lens), n_pos, device="cuda")
    csa2.csa2_index_score(q, s, w, flat[2], flat[3], c.n_visible, want)
    counters = torch.zeros(2 * len(lens), dtype=torch.int32, device="cuda") if claimed else None
    for _ in range(2):
        got = torch.full_like(want, 5.0)
        csa2.csa2_paged_index_score(q, s, w, c.ik_data, c.ik_scale, c.table, c.n_visible, got, tile_counters=counters)
        assert torch.equal(got, want)
        assert counters is None or not counters.any()
    assert csa2.csa2_get_last_error() == 0


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("claimed", [False, True])
@pytest.mark.parametrize("lens,n_pos", [
    ([0, 1, 12000, 11999, 128, 4097, 9000, 12000, 640], 12000),  # CTAs in proportion to lengths
    ([0, 5, 30001], 40003),  # one long sequence, and room behind it
    ([200 + 3 * (i % 61) for i in range(500)], 391),  # more sequences than CTAs in a wave
    ([3000, 0, 9000], 2777),  # more entries than scores are asked for
])
def test_scores_of_many_tiles_equal_the_flat_scan(csa2, page, claimed, lens, n_pos):
    c = Cache(csa2, lens, page, 26 + page)
    q, s, w = queries(csa2, gen(27), len(lens))
    flat = c.flat_planes()
    cap = flat[2].shape[1]
    want = torch.full((len(lens), n_pos), -float("inf"), device="cuda")
    least = torch.empty(len(lens), min(n_pos, cap), device="cuda")
    csa2.csa2_index_score(q, s, w, flat[2], flat[3], c.n_visible, least)
    want[:, :least.shape[1]] = least
    places = -(-n_pos // page)
    table = torch.full((len(lens), max(places, c.table.shape[1])), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    counters = torch.zeros(2 * len(lens), dtype=torch.int32, device="cuda") if claimed else None
    for _ in range(2):
        got = torch.full_like(want, 5.0)
        csa2.csa2_paged_index_score(q, s, w, c.ik_data, c.ik_scale, table, c.n_visible, got, tile_counters=counters)
        assert torch.equal(got, want)
        assert counters is None or not counters.any()
    assert csa2.csa2_get_last_error() == 0


def test_scores_with_a_negative_counter(csa2):
    """A counter that was not cleared is reported, and no page is looked up before the table."""
    c = Cache(csa2, [9000] * 8, 64, 28)
    q, s, w = queries(csa2, gen(29), 8)
    counters = torch.zeros(16, dtype=torch.int32, device="cuda")
    counters[0::2] = -(1 << 30)
    got = torch.empty(8, 9000, device="cuda")
    csa2.csa2_paged_index_score(q, s, w, c.ik_data, c.ik_scale, c.table, c.n_visible, got, tile_counters=counters)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR


def test_scores_against_64_bits(csa2):
    lens = [300, 41]
    c = Cache(csa2, lens, 32, 22)
    q, s, w = queries(csa2, gen(23), 2)
    got = torch.empty(2, 300, device="cuda")
    csa2.csa2_paged_index_score(q, s, w, c.ik_data, c.ik_scale, c.table, c.n_visible, got)
    qf = torch.empty(2, 32, 128, device="cuda")
    csa2.csa2_dequant_mxfp4(q, s, qf)
    for b, n in enumerate(lens):
        kf = torch.empty(n, 128, device="cuda")
        csa2.csa2_dequant_mxfp4(c.ik_data.view(-1, 64)[c.rows[b]].contiguous(), c.ik_scale.view(-1, 4)[c.rows[b]].contiguous(), kf)
        ref = w[b].double() @ torch.relu(qf[b].double() @ kf.double().T)
        assert torch.all((got[b, :n].double() - ref).abs() <= 1e-5 * ref + 1e-6 * ref.max())
        assert torch.all(got[b, n:] == -float("inf"))


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("claimed", [False, True])
def test_scores_of_missing_pages(csa2, page, claimed):
    """A page outside the pool scores -inf and is reported; its neighbours are not touched by it."""
    lens = [1000, 600]
    c = Cache(csa2, lens, page, 24)
    q, s, w = queries(csa2, gen(25), 2)
    want = torch.empty(2, 1000, device="cuda")
    csa2.csa2_paged_index_score(q, s, w, c.ik_data, c.ik_scale, c.table, c.n_visible, want)
    assert csa2.csa2_get_last_error() == 0
    c.table[0, 2], c.table[1, 0], c.table[0, 999 // page] = c.pages, -1, 1 << 30
    for b, at in ((0, 2), (1, 0), (0, 999 // page)):
        want[b, at * page:(at + 1) * page] = -float("inf")
    counters = torch.zeros(4, dtype=torch.int32, device="cuda") if claimed else None
    got = torch.empty_like(want)
    csa2.csa2_paged_index_score(q, s, w, c.ik_data, c.ik_scale, c.table, c.n_visible, got, tile_counters=counters)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    assert torch.equal(got, want)


# ---- sparse attention -------------------------------------------------------------------


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("B,L,k,n_swa", [(1, 1, 512, 128), (5, 4, 512, 128), (3, 2, 100, 37), (40, 1, 512, 0), (2, 1, 0, 16)])
def test_sparse_attention_equals_the_flat_call(csa2, page, B, L, k, n_swa):
    g = gen(B + k)
    lens = [max(1, 700 - 61 * i) if i < 11 else 90 + i for i in range(B)]
    c = Cache(csa2, lens, page, 30 + B)
    q = normal(g, B, L, 64, 512, scale=512 ** -0.5)
    swa = csa2.pack_fp8(normal(g, B, L, n_swa, 512)) if n_swa else None
    idx = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        pick = torch.randperm(n, generator=g, device="cuda")[:k].sort().values
        idx[b, :pick.numel()] = pick.int()
    flat = c.flat_planes()
    res = []
    for paged in (False, True):
        out, f32 = torch.empty_like(q), torch.empty(q.shape, device="cuda")
        lse = torch.empty(B, L, 64, device="cuda")
        if paged:
            csa2.csa2_paged_sparse_attn_decode(q, c.kv_data, c.kv_scale, c.table, c.n_visible, idx, swa, out,
                                               csa2.paged_sparse_attn_workspace(B, L, k, n_swa), out_f32=f32, lse=lse)
        else:
            # (the flat binding hands an empty idx over as a null pointer, which it refuses)
            one = idx if k else torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
            csa2.csa2_sparse_attn_decode(q, flat[0], flat[1], c.n_visible, one, swa, out,
                                         csa2.attn_workspace(B * L, max(k, 1), n_swa), out_f32=f32, lse=lse)
        res.append((out, f32, lse))
    assert csa2.csa2_get_last_error() == 0
    if k:
        for a, b in zip(*res):
            assert torch.equal(a, b)
    else:  # an empty list and a list of one empty place: the same rows in another plan
        assert torch.allclose(res[0][1], res[1][1], rtol=0, atol=2.0 ** -10)


@pytest.mark.parametrize("form,B,L,k,n_swa", [("reuse", 3, 4, 512, 128)] + [
    (form, *shape) for form in ("paged", "flat")
    for shape in ((1, 1, 512, 128), (3, 4, 512, 128), (20, 1, 128, 128), (2, 1, 128, 512), (40, 1, 512, 16))])
def test_selected_attention_calls_in_a_row_share_a_workspace(csa2, form, B, L, k, n_swa):
    """Layer after layer with one workspace, eager and captured: a call may not write its partials while the call before it still
    reads its own (it starts on its window before that call has ended)."""
    g = gen(106)
    lens = [700 - 10 * b for b in range(B)]
    c = Cache(csa2, lens, 64, 107)
    flat = c.flat_planes()
    idx = torch.stack([torch.randperm(min(lens), generator=g, device="cuda")[:k].sort().values for _ in range(B)]).int()
    if idx.shape[1] < k:
        idx = torch.cat([idx, torch.full((B, k - idx.shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    idx = idx.contiguous()
    layers = [(normal(g, B, L, 64, 512, scale=512 ** -0.5), csa2.pack_fp8(normal(g, B, L, n_swa, 512, scale=i + 1.0))) for i in range(4)]
    ws = csa2.paged_sparse_attn_workspace(B, L, k, n_swa)

    def call(i, out):
        q, swa = layers[i]
        if form == "paged":
            csa2.csa2_paged_sparse_attn_decode(q, c.kv_data, c.kv_scale, c.table, c.n_visible, idx, swa, out, ws)
        elif form == "flat":
            csa2.csa2_sparse_attn_decode(q, flat[0], flat[1], c.n_visible, idx, swa, out, ws)
        else:
            csa2.csa2_sparse_attn_reuse(q, flat[0], flat[1], c.n_visible, idx, swa, out, ws)

    outs = [torch.empty_like(q) for q, _ in layers]
    for i, o in enumerate(outs):
        call(i, o)
        torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, o in enumerate(outs):
            call(i, o)
    for n in range(40):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        if n % 2:
            graph.replay()
        else:
            for i, o in enumerate(outs):
                call(i, o)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (n, i)
    assert csa2.csa2_get_last_error() == 0


def test_sparse_attention_skips_what_is_not_there(csa2):
    """Entries at or past n_visible and entries of missing pages are left out and reported."""
    g = gen(33)
    c = Cache(csa2, [200, 64], 16, 34)
    q = normal(g, 2, 1, 64, 512, scale=512 ** -0.5)
    idx = ints([[0, 5, 17, 199, 200], [3, 63, 64, 1 << 30, -1]])
    kept = ints([[0, 5, -1, 199, -1], [3, 63, -1, -1, -1]])
    ws = csa2.paged_sparse_attn_workspace(2, 1, 5, 0)
    want, got = torch.empty_like(q), torch.empty_like(q)
    csa2.csa2_paged_sparse_attn_decode(q, c.kv_data, c.kv_scale, c.table, c.n_visible, kept, None, want, ws)
    assert csa2.csa2_get_last_error() == 0
    c.table[0, 1] = -7
    csa2.csa2_paged_sparse_attn_decode(q, c.kv_data, c.kv_scale, c.table, c.n_visible, idx, None, got, ws)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    assert torch.equal(got, want)


# ---- dense attention ---------------------------------------------------------------------


def dense_reference(q, rows, scale):
    """(out, lse, the sums and the score error that the tolerance is made of) of q [64, 512] over rows [n, 512]."""
    q = q.double()
    if not rows.shape[0]:
        z = torch.zeros(64, 512, dtype=torch.float64, device="cuda")
        return z, torch.full((64,), -float("inf"), dtype=torch.float64, device="cuda"), z, 0.0
    x = scale * (q @ rows.T)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    d = 512 * 2.0 ** -24 * abs(scale) * float((q.abs() @ rows.abs().T).max())
    return p @ rows, lse, p @ rows.abs(), d


def run_dense(csa2, c, q, cu=None, causal=True, scale=1.0, fill=7.0, ws=None):
    n = q.shape[0]
    out = torch.full_like(q, fill)
    f32 = torch.full(q.shape, fill, device="cuda")
    lse = torch.full((n, 64), fill, device="cuda")
    ws = csa2.paged_attn_workspace(n, len(c.lens)) if ws is None else ws
    csa2.csa2_paged_attn(q, c.kv_data, c.kv_scale, c.table, c.n_visible, out, ws, cu_q=cu, causal=causal, out_f32=f32, lse=lse,
                         sm_scale=scale)
    return out, f32, lse


def check_dense(csa2, c, q, runs, first, causal, scale, got):
    out, f32, lse = got
    at = first
    for b, T in enumerate(runs):
        rows = c.latents(csa2, b)
        for j in range(T):
            n = c.lens[b]
            seen = max(0, n - T + 1 + j) if causal else n
            o, l, a, d = dense_reference(q[at], rows[:seen], scale)
            err = (f32[at].double() - o).abs()
            tol = (2.0 ** -11 + 3 * d + 2.0 ** -18) * a + 1e-30
            assert torch.all(err <= tol), (b, j, seen, float((err / tol).max()))
            if seen:
                assert torch.all((lse[at].double() - l).abs() <= d + 2.0 ** -18 * (1 + l.abs())), (b, j)
            else:
                assert torch.all(lse[at] == -float("inf"))
            at += 1
    mid = slice(first, at)
    assert torch.equal(out[mid], f32[mid].bfloat16())
    assert torch.all(out[:first] == 7.0) and torch.all(out[at:] == 7.0) and torch.all(lse[at:] == 7.0)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 127, 128, 129, 255, 257, 1000])
def test_dense_one_token(csa2, n, page):
    c = Cache(csa2, [n], page, 40 + n, unused=1 << 30)
    q = normal(gen(n), 1, 64, 512, scale=512 ** -0.5)
    got = run_dense(csa2, c, q)
    assert csa2.csa2_get_last_error() == 0
    check_dense(csa2, c, q, [1], 0, True, 1.0, got)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("runs,lens,page", [
    ([1, 1, 1, 1], [4097, 1, 130, 999], 64),
    ([3, 0, 1, 4, 2], [300, 50, 0, 2, 513], 16),          # no tokens, no entries, tokens before the first entry
    ([40, 17], [40, 300], 128),                          # prompts with and without a past
    ([160, 1, 33], [161, 5000, 20], 32),                 # more tokens than SMs, and a token over several of them
    ([0, 0, 0], [7, 8, 9], 16)])
def test_dense_ragged(csa2, runs, lens, page, causal):
    c = Cache(csa2, lens, page, 50 + len(runs))
    g = gen(51)
    first, behind = 2, 3
    q = normal(g, first + sum(runs) + behind, 64, 512, scale=512 ** -0.5)
    got = run_dense(csa2, c, q, cu=starts(runs, first), causal=causal)
    assert csa2.csa2_get_last_error() == 0
    check_dense(csa2, c, q, runs, first, causal, 1.0, got)


@pytest.mark.parametrize("scale", [1.0, 0.05, -0.3, 0.0])
def test_dense_scores_that_rise(csa2, scale):
    """Scores that grow along the entries move the reference of the weights again and again; some heads fall instead."""
    n = 1500
    c = Cache(csa2, [n], 64, 60)
    rows = c.latents(csa2, 0)
    g = gen(61)
    q = normal(g, 2, 64, 512, scale=0.3)
    with torch.no_grad():  # entry j looks like the queries' common direction, ever more so
        base = normal(g, 512).float()
        x = (torch.randn(n, 512, generator=g, device="cuda") + base * torch.linspace(-2, 2, n, device="cuda")[:, None]).bfloat16()
        q = (q.float() + torch.where(torch.arange(64, device="cuda") % 3 == 0, -0.05, 0.05)[None, :, None] * base).bfloat16()
    d, s = csa2.pack_kv_fp4(x)
    c.kv_data.view(-1, 256)[c.rows[0]] = d
    c.kv_scale.view(-1, 32)[c.rows[0]] = s
    got = run_dense(csa2, c, q, scale=scale)
    assert csa2.csa2_get_last_error() == 0
    check_dense(csa2, c, q, [2], 0, True, scale, got)


def test_dense_weights_far_below_the_largest(csa2):
    """One entry takes nearly all of a head's weight and comes first: the others' sum is still there. Their weights are 2^-22
    of the largest and below, yet each is rounded relative to itself."""
    n = 2000
    c = Cache(csa2, [n], 128, 62)
    x = torch.zeros(n, 512, device="cuda")
    x[0, 0] = 6.0          # the first entry
    x[1:, 1] = 6.0         # the others, seen in channel 1
    d, s = csa2.pack_kv_fp4(x.bfloat16())
    c.kv_data.view(-1, 256)[c.rows[0]] = d
    c.kv_scale.view(-1, 32)[c.rows[0]] = s
    q = torch.zeros(1, 64, 512, device="cuda")
    q[0, :, 0] = torch.linspace(0.5, 2.5, 64)  # scores of the first entry: 3 .. 15
    got = run_dense(csa2, c, q.bfloat16())
    check_dense(csa2, c, q.bfloat16(), [1], 0, True, 1.0, got)


def test_dense_queries_of_very_different_sizes(csa2):
    c = Cache(csa2, [333], 16, 63)
    q = normal(gen(64), 1, 64, 512, scale=512 ** -0.5)
    q[0, 3] = 0
    q[0, 5] *= 1e-30
    q[0, 6] *= 1e-6
    q[0, 7] *= 30
    got = run_dense(csa2, c, q)
    check_dense(csa2, c, q, [1], 0, True, 1.0, got)


@pytest.mark.parametrize("e", [124, 110, -100])
def test_attention_of_queries_at_the_ends_of_their_type(csa2, e):
    """Queries times 2^e with sm_scale 2^-e are the same scores to the last bit, dense, selected and on flat planes."""
    c = Cache(csa2, [400, 33], 16, 92)
    q = normal(gen(93), 2, 64, 512, scale=512 ** -0.5)
    q = torch.where(q.abs() < 2.0 ** -20, 0, q)  # (nothing becomes subnormal)
    far = (q.double() * 2.0 ** e).bfloat16()
    assert torch.equal(far.double() * 2.0 ** -e, q.double())
    idx = ints([[0, 5, 17, 399], [3, 32, -1, -1]])
    swa = csa2.pack_fp8(normal(gen(94), 2, 1, 16, 512))
    flat = c.flat_planes()
    res = []
    for x, scale in ((q, 1.0), (far, 2.0 ** -e)):
        dense = run_dense(csa2, c, x, scale=scale)
        x = x[:, None].contiguous()
        o1, o2, l1 = torch.empty_like(x), torch.empty_like(x), torch.empty(2, 1, 64, device="cuda")
        csa2.csa2_paged_sparse_attn_decode(x, c.kv_data, c.kv_scale, c.table, c.n_visible, idx, swa, o1,
                                           csa2.paged_sparse_attn_workspace(2, 1, 4, 16), lse=l1, sm_scale=scale)
        csa2.csa2_sparse_attn_decode(x, flat[0], flat[1], c.n_visible, idx, swa, o2, csa2.attn_workspace(2, 4, 16),
                                     sm_scale=scale)
        res.append((*dense, o1, l1, o2))
    assert csa2.csa2_get_last_error() == 0
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [0, 31, 32, 63])
def test_dense_heads_with_scores_past_32_bits(csa2, bad):
    """A head whose scores all pass fp32's range downwards leaves the other heads of its token as they are, whichever it is:
    the first tile sets their references although that head has no maximum."""
    n = 40000  # (several tiles to an SM)
    c = Cache(csa2, [n], 64, 99)
    x = normal(gen(100), n, 512)
    x[:, 0] = 6.0
    x *= torch.linspace(0.5, 3.0, n, device="cuda").flip(0)[:, None].bfloat16()  # (the maxima change)
    d, s = csa2.pack_kv_fp4(x)
    c.kv_data.view(-1, 256)[c.rows[0]] = d
    c.kv_scale.view(-1, 32)[c.rows[0]] = s.view(torch.uint8)
    q = normal(gen(101), 2, 64, 512, scale=0.2)
    want = run_dense(csa2, c, q)
    q[:, bad] = 0
    q[:, bad, 0] = -3e38
    got = run_dense(csa2, c, q)
    assert csa2.csa2_get_last_error() == 0
    others = [h for h in range(64) if h != bad]
    for a, b in zip(got, want):
        assert torch.equal(a[:, others], b[:, others])
    check = [t[:, others] for t in got]
    rows = c.latents(csa2, 0)
    for j in range(2):
        o, l, a, err = dense_reference(q[j][others], rows[:n - 1 + j], 1.0)
        assert torch.all((check[1][j].double() - o).abs() <= (2.0 ** -11 + 3 * err + 2.0 ** -18) * a + 1e-30)


def test_dense_missing_pages_and_bad_counts(csa2):
    c = Cache(csa2, [500, 300, 200, 100], 16, 65, most=40)
    g = gen(66)
    q = normal(g, 4, 64, 512, scale=512 ** -0.5)
    want = run_dense(csa2, c, q)
    keep = c.table.clone()
    # sequence 0 loses a page in a tile's middle, sequence 1 its whole first tile
    c.table[0, 9] = -1
    c.table[1, :8] = c.pages + torch.arange(8, device="cuda").int()
    got = run_dense(csa2, c, q)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    gone = [set(range(144, 160)), set(range(128)), set(), set()]
    for b in range(4):
        rows = c.latents(csa2, b)
        left = torch.tensor([i for i in range(c.lens[b]) if i not in gone[b]], device="cuda")
        o, l, a, d = dense_reference(q[b], rows[left], 1.0)
        assert torch.all((got[1][b].double() - o).abs() <= (2.0 ** -11 + 3 * d + 2.0 ** -18) * a), b
        assert torch.all((got[2][b].double() - l).abs() <= d + 2.0 ** -18 * (1 + l.abs())), b
    # counts that are negative or above the table's places: passed over
    c.table.copy_(keep)
    c.n_visible = ints([500, -1, 40 * 16 + 1, 100])
    got = run_dense(csa2, c, q)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    for b in (1, 2):
        assert torch.all(got[0][b] == 7.0) and torch.all(got[2][b] == 7.0)
    for b in (0, 3):
        rows = c.latents(csa2, b)
        o, l, a, d = dense_reference(q[b], rows, 1.0)
        assert torch.all((got[1][b].double() - o).abs() <= (2.0 ** -11 + 3 * d + 2.0 ** -18) * a), b
    # a run outside the rows: that sequence is passed over
    c.n_visible = ints([500, 300, 200, 100])
    got = run_dense(csa2, c, q, cu=ints([0, 1, 9, 2, 3]))
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    assert torch.all(got[0][3] == 7.0)
    # the same again, clean
    again = run_dense(csa2, c, q)
    assert csa2.csa2_get_last_error() == 0
    for a, b in zip(again, want):
        assert torch.equal(a, b)


def test_dense_same_bits_twice_and_without_the_optional_outputs(csa2):
    c = Cache(csa2, [3000, 10, 700], 64, 67)
    q = normal(gen(68), 30, 64, 512, scale=512 ** -0.5)
    cu = starts([9, 20, 1])
    a = run_dense(csa2, c, q, cu=cu)
    b = run_dense(csa2, c, q, cu=cu)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    out = torch.empty_like(q)
    csa2.csa2_paged_attn(q, c.kv_data, c.kv_scale, c.table, c.n_visible, out, csa2.paged_attn_workspace(30, 3), cu_q=cu)
    assert torch.equal(out, a[0])


def test_dense_many_sequences(csa2):
    """More sequences than a block has threads; most of them short, some empty."""
    lens = [(37 * i) % 90 for i in range(1300)]
    c = Cache(csa2, [max(lens)] * 2, 16, 69)  # every sequence shares the pages of these two
    table = c.table[torch.arange(1300, device="cuda") % 2].contiguous()
    q = normal(gen(70), 1300, 64, 512, scale=512 ** -0.5)
    out, f32 = torch.empty_like(q), torch.empty(q.shape, device="cuda")
    csa2.csa2_paged_attn(q, c.kv_data, c.kv_scale, table, ints(lens), out, csa2.paged_attn_workspace(1300, 1300), out_f32=f32)
    assert csa2.csa2_get_last_error() == 0
    rows = [c.latents(csa2, 0), c.latents(csa2, 1)]
    for i in list(range(0, 1300, 97)) + [511, 512, 513, 1023, 1024, 1299]:
        o, _, a, d = dense_reference(q[i], rows[i % 2][:lens[i]], 1.0)
        assert torch.all((f32[i].double() - o).abs() <= (2.0 ** -11 + 3 * d + 2.0 ** -18) * a + 1e-30), i


def test_dense_many_ragged_sequences(csa2):
    """More sequences than threads, zero to five tokens each, and two with counts that are refused."""
    B = 1100
    runs = [(7 * i) % 6 for i in range(B)]
    lens = [(53 * i) % 400 for i in range(B)]
    bad = {17: -1, 1043: 401}
    c = Cache(csa2, [400] * 2, 16, 71)  # every sequence shares the pages of these two
    table = c.table[torch.arange(B, device="cuda") % 2].contiguous()
    n = sum(runs)
    q = normal(gen(72), n, 64, 512, scale=512 ** -0.5)
    out, f32 = torch.full_like(q, 7.0), torch.full(q.shape, 7.0, device="cuda")
    csa2.csa2_paged_attn(q, c.kv_data, c.kv_scale, table, ints([bad.get(i, v) for i, v in enumerate(lens)]), out,
                         csa2.paged_attn_workspace(n, B), cu_q=starts(runs), out_f32=f32)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR
    rows = [c.latents(csa2, 0), c.latents(csa2, 1)]
    at = 0
    for b, T in enumerate(runs):
        for j in range(T):
            if b in bad:
                assert torch.all(f32[at] == 7.0) and torch.all(out[at] == 7.0)
            elif b % 53 == 0 or b > B - 4 or 894 <= b <= 898 or b in (16, 18, 1042, 1044):
                o, _, a, d = dense_reference(q[at], rows[b % 2][:max(0, lens[b] - T + 1 + j)], 1.0)
                assert torch.all((f32[at].double() - o).abs() <= (2.0 ** -11 + 3 * d + 2.0 ** -18) * a + 1e-30), (b, j)
            at += 1


@pytest.mark.parametrize("runs,past", [([300, 1, 0, 517, 2], 0), ([90, 700], 70), ([1] * 400, 3)])
def test_dense_prompts_and_short_steps(csa2, runs, past):
    """Tokens of one to seven tiles: runs of an SM that begin and end inside tokens and between them."""
    lens = [T + (past if T > 1 else 5 * i + past) for i, T in enumerate(runs)]
    c = Cache(csa2, lens, 32, 73 + past)
    q = normal(gen(74), sum(runs), 64, 512, scale=512 ** -0.5)
    got = run_dense(csa2, c, q, cu=starts(runs))
    assert csa2.csa2_get_last_error() == 0
    check_dense(csa2, c, q, runs, 0, True, 1.0, got)


def test_dense_two_calls_at_once(csa2):
    """Two streams with a workspace each, many times over, give the bits of the calls alone."""
    calls = []
    for i, (runs, lens) in enumerate([([4, 1, 9], [3000, 20, 700]), ([1] * 40, [150 + 7 * j for j in range(40)])]):
        c = Cache(csa2, lens, 64, 75 + i)
        q = normal(gen(77 + i), sum(runs), 64, 512, scale=512 ** -0.5)
        alone = run_dense(csa2, c, q, cu=starts(runs))
        outs = torch.empty_like(q), torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
        calls.append((c, q, starts(runs), alone, outs, csa2.paged_attn_workspace(q.shape[0], len(runs)), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, cu, _, (out, f32, lse), ws, stream in calls:
            csa2.csa2_paged_attn(q, c.kv_data, c.kv_scale, c.table, c.n_visible, out, ws, cu_q=cu, out_f32=f32, lse=lse,
                                 stream=stream)
    torch.cuda.synchronize()
    assert csa2.csa2_get_last_error() == 0
    for _, _, _, alone, outs, _, _ in calls:
        for x, y in zip(alone, outs):
            assert torch.equal(x, y)


def test_dense_rows_past_32_bits(csa2):
    """Pages whose bytes lie more than 2^32 behind the plane's start."""
    page, n = 128, 700
    pages = (1 << 24) // page + 8                       # 256 bytes a row: 4 GiB and a little
    small = Cache(csa2, [n], page, 71)
    data = torch.zeros(pages, page, 256, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(pages, page, 32, dtype=torch.uint8, device="cuda")
    far = torch.arange(pages - 6, pages, dtype=torch.int32, device="cuda")[None]
    data[far[0].long()] = small.kv_data[small.table[0].long()]
    scale[far[0].long()] = small.kv_scale[small.table[0].long()]
    q = normal(gen(72), 2, 64, 512, scale=512 ** -0.5)
    want = run_dense(csa2, small, q)
    out = torch.empty_like(q)
    csa2.csa2_paged_attn(q, data, scale, far, small.n_visible, out, csa2.paged_attn_workspace(2, 1))
    assert csa2.csa2_get_last_error() == 0
    assert torch.equal(out, want[0])
    idx = torch.arange(512, dtype=torch.int32, device="cuda")[None]
    o1, o2 = torch.empty(1, 1, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, 64, 512, dtype=torch.bfloat16, device="cuda")
    ws = csa2.paged_sparse_attn_workspace(1, 1, 512, 0)
    csa2.csa2_paged_sparse_attn_decode(q[:1, None].contiguous(), data, scale, far, small.n_visible, idx, None, o1, ws)
    csa2.csa2_paged_sparse_attn_decode(q[:1, None].contiguous(), small.kv_data, small.kv_scale, small.table, small.n_visible, idx,
                                       None, o2, ws)
    assert torch.equal(o1, o2)


def test_dense_joins_the_window_by_merge(csa2):
    """All entries and the FP8 window in one softmax: the dense part and the window's part merged equal the sparse call that
    selects every entry."""
    lens = [300, 77]
    c = Cache(csa2, lens, 64, 73)
    g = gen(74)
    q = normal(g, 2, 64, 512, scale=512 ** -0.5)
    swa = csa2.pack_fp8(normal(g, 2, 1, 128, 512))
    _, f1, l1 = run_dense(csa2, c, q)
    none = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    f2, l2, o = torch.empty(2, 1, 64, 512, device="cuda"), torch.empty(2, 1, 64, device="cuda"), torch.empty(2, 1, 64, 512, dtype=torch.bfloat16, device="cuda")
    csa2.csa2_paged_sparse_attn_decode(q[:, None].contiguous(), c.kv_data, c.kv_scale, c.table, c.n_visible, none, swa, o,
                                       csa2.paged_sparse_attn_workspace(2, 1, 1, 128), out_f32=f2, lse=l2)
    merged, mf = torch.empty_like(q), torch.empty(q.shape, device="cuda")
    csa2.csa2_attn_merge(torch.stack([f1, f2[:, 0]]), torch.stack([l1, l2[:, 0]]), merged, out_f32=mf)
    window = torch.empty(2, 128, 512, dtype=torch.bfloat16, device="cuda")
    csa2.csa2_unpack_fp8_e4m3(swa, window)
    for b in range(2):
        rows = torch.cat([c.latents(csa2, b), window[b].double()])
        ref, _, a, d = dense_reference(q[b], rows, 1.0)
        # the merge adds its own fp32 weights: 2^-18 once more
        assert torch.all((mf[b].double() - ref).abs() <= (2.0 ** -11 + 5 * d + 2.0 ** -17) * a)


def test_a_pool_without_pages(csa2):
    """Sequences without entries over a pool that has none; and entries that are nowhere."""
    planes = [torch.empty(0, 16, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    g = gen(102)
    q = normal(g, 3, 64, 512, scale=512 ** -0.5)
    qi, qs, w = queries(csa2, g, 2)
    swa = csa2.pack_fp8(normal(g, 2, 1, 16, 512))
    idx = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    sq = q[:2, None].contiguous()
    alone = torch.empty_like(sq)
    flat = torch.zeros(2, 128, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 128, 32, dtype=torch.uint8, device="cuda")
    csa2.csa2_sparse_attn_decode(sq, *flat, ints([0, 0]), idx, swa, alone, csa2.attn_workspace(2, 4, 16))
    for lens, status in (([0, 0], 0), ([5, 40], DEVICE_ERROR)):
        nv = ints(lens)
        out, lse = torch.full_like(q, 7.0), torch.full((3, 64), 7.0, device="cuda")
        csa2.csa2_paged_attn(q, planes[0], planes[1], table, nv, out, csa2.paged_attn_workspace(3, 2), cu_q=ints([0, 2, 3]), lse=lse)
        assert csa2.csa2_get_last_error() == status
        assert torch.all(out == 0) and torch.all(lse == -float("inf"))
        scores = torch.full((2, 48), 7.0, device="cuda")
        csa2.csa2_paged_index_score(qi, qs, w, planes[2], planes[3], table, nv, scores)
        assert csa2.csa2_get_last_error() == status
        assert torch.all(scores == -float("inf"))
        pick = torch.arange(4, dtype=torch.int32, device="cuda").repeat(2, 1) if status else idx
        got = torch.full_like(sq, 7.0)
        csa2.csa2_paged_sparse_attn_decode(sq, planes[0], planes[1], table, nv, pick, swa, got,
                                           csa2.paged_sparse_attn_workspace(2, 1, 4, 16))
        assert csa2.csa2_get_last_error() == status
        assert torch.equal(got, alone)
    kv, ik = normal(g, 2, 512), normal(g, 2, 128)
    after = torch.empty(2, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_kv_append(kv[:0], ik[:0], *planes, table, ints([0, 0]), after)
    assert csa2.csa2_get_last_error() == 0 and after.tolist() == [0, 0]
    csa2.csa2_paged_kv_append(kv, ik, *planes, table, ints([0, 0]), after)
    assert csa2.csa2_get_last_error() == DEVICE_ERROR and after.tolist() == [1, 1]


# ---- a server's use of them ------------------------------------------------------------------


def test_prompt_then_steps(csa2):
    """Prompts appended in two chunks, then decode steps: append, scores, Top-K, sparse and dense attention, queries and outputs
    rotated. The cache equals one packed at once, the selections equal the flat path's, attention equals its definition."""
    g = gen(80)
    B, page, most = 3, 32, 8
    prompt, steps = [70, 1, 133], 4
    total = [p + steps for p in prompt]
    table, pages = tables([most * page] * B, page, g)
    planes = [torch.zeros(pages, page, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)]
    rope = angles(most * page, 64)
    xs = [normal(g, n, 512) for n in total]
    ks = [normal(g, n, 128) for n in total]
    nv = torch.zeros(B, dtype=torch.int32, device="cuda")
    done = [0] * B

    def append(runs):
        kv = torch.cat([x[d:d + r] for x, d, r in zip(xs, done, runs)])
        ik = torch.cat([x[d:d + r] for x, d, r in zip(ks, done, runs)])
        csa2.csa2_paged_kv_append(kv, ik, *planes, table, nv, nv, cu_tokens=starts(runs), rope=rope, interleaved=True)
        for b, r in enumerate(runs):
            done[b] += r

    append([60, 1, 33])
    append([10, 0, 100])
    counters = torch.zeros(2 * B, dtype=torch.int32, device="cuda")
    k = 64
    for _ in range(steps):
        append([1, 1, 1])
        assert nv.tolist() == done
        q = normal(g, B, 64, 512, scale=512 ** -0.5)
        turned = torch.empty_like(q)
        csa2.csa2_rope(q, rope, nv - 1, turned, interleaved=True)
        qi, qs, w = queries(csa2, g, B)
        scores = torch.empty(B, most * page, device="cuda")
        csa2.csa2_paged_index_score(qi, qs, w, planes[2], planes[3], table, nv, scores, tile_counters=counters)
        idx = torch.empty(B, k, dtype=torch.int32, device="cuda")
        csa2.csa2_topk(scores, k, idx, csa2.topk_workspace(B, most * page, k), n_valid=nv)
        sparse, s32 = torch.empty(B, 1, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, 64, 512, device="cuda")
        csa2.csa2_paged_sparse_attn_decode(turned[:, None].contiguous(), planes[0], planes[1], table, nv, idx, None, sparse,
                                           csa2.paged_sparse_attn_workspace(B, 1, k, 0), out_f32=s32)
        dense, d32 = torch.empty_like(q), torch.empty(q.shape, device="cuda")
        csa2.csa2_paged_attn(turned, planes[0], planes[1], table, nv, dense, csa2.paged_attn_workspace(B, B), out_f32=d32)
        back = torch.empty_like(dense)
        csa2.csa2_rope(dense, rope, nv - 1, back, interleaved=True, inverse=True)
        assert csa2.csa2_get_last_error() == 0
        for b in range(B):
            n = done[b]
            e = torch.arange(n, device="cuda")
            ref_d, ref_s = oracle.pack_kv_fp4(rotated(xs[b][:n], rope, e, True).float().cpu().numpy())
            rows = rows_of(table, b, n, page)
            assert torch.equal(planes[0].view(-1, 256)[rows].cpu(), torch.from_numpy(ref_d))
            assert torch.equal(planes[1].view(-1, 32)[rows].cpu(), torch.from_numpy(ref_s))
            ik_d, ik_s = oracle.quant_mxfp4(rotated(ks[b][:n], rope, e, True).float().cpu().numpy())
            s32_ref = oracle.index_score(qi[b].cpu().numpy(), qs[b].cpu().numpy(), w[b].cpu().numpy(), ik_d, ik_s)[0]
            from helpers import check_topk
            check_topk(s32_ref, idx[b].cpu().numpy(), k)
            lat = torch.empty(n, 512, dtype=torch.bfloat16, device="cuda")
            csa2.csa2_unpack_kv_fp4(planes[0].view(-1, 256)[rows].contiguous(), planes[1].view(-1, 32)[rows].contiguous(), lat)
            lat = lat.double()
            o, _, a, d = dense_reference(turned[b], lat, 1.0)
            assert torch.all((d32[b].double() - o).abs() <= (2.0 ** -11 + 3 * d + 2.0 ** -18) * a)
            pick = idx[b][idx[b] >= 0].long()
            o, _, a, d = dense_reference(turned[b], lat[pick], 1.0)
            assert torch.all((s32[b, 0].double() - o).abs() <= (2.0 ** -11 + 3 * d + 2.0 ** -18) * a)
        want = rotated(dense, rope, nv - 1, True, inverse=True)
        assert torch.all((back.double() - want).abs() <= want.abs() * 2.0 ** -8 * (1 + 2.0 ** -14) + 1e-38)


def test_captured_steps_replay(csa2):
    """A captured decode step (append in place, scores, Top-K, both attentions) replayed as the sequences grow equals the eager
    steps; the graph holds a workspace of its own while another call runs on another stream with its own."""
    g = gen(81)
    B, page, most, k = 4, 16, 20, 32
    past = [3, 0, 200, 31]
    c_table, pages = tables([most * page] * B, page, g)
    rope = angles(most * page, 32)

    def fresh():
        return [torch.zeros(pages, page, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 64, 4)], ints([0] * B)

    kv0, ik0 = normal(g, sum(past), 512), normal(g, sum(past), 128)
    steps = [(normal(g, B, 512), normal(g, B, 128), normal(g, B, 64, 512, scale=512 ** -0.5)) for _ in range(5)]
    qi, qs, w = queries(csa2, g, B)

    class Step:
        def __init__(self):
            self.planes, self.nv = fresh()
            csa2.csa2_paged_kv_append(kv0, ik0, *self.planes, c_table, self.nv, self.nv, cu_tokens=starts(past), rope=rope)
            self.kv, self.ik, self.q = (torch.empty_like(t) for t in steps[0])
            self.scores = torch.empty(B, most * page, device="cuda")
            self.idx = torch.empty(B, k, dtype=torch.int32, device="cuda")
            self.sparse, self.dense = torch.empty(B, 1, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty_like(self.q)
            self.lse = torch.empty(B, 64, device="cuda")
            self.ws1, self.ws2 = csa2.topk_workspace(B, most * page, k), csa2.paged_sparse_attn_workspace(B, 1, k, 0)
            self.ws3 = csa2.paged_attn_workspace(B, B)
            self.counters = torch.zeros(2 * B, dtype=torch.int32, device="cuda")

        def load(self, i):
            for to, x in zip((self.kv, self.ik, self.q), steps[i]):
                to.copy_(x)

        def run(self):
            csa2.csa2_paged_kv_append(self.kv, self.ik, *self.planes, c_table, self.nv, self.nv, rope=rope)
            csa2.csa2_paged_index_score(qi, qs, w, self.planes[2], self.planes[3], c_table, self.nv, self.scores,
                                        tile_counters=self.counters)
            csa2.csa2_topk(self.scores, k, self.idx, self.ws1, n_valid=self.nv)
            csa2.csa2_paged_sparse_attn_decode(self.q.view(B, 1, 64, 512), self.planes[0], self.planes[1], c_table, self.nv, self.idx,
                                               None, self.sparse, self.ws2)
            csa2.csa2_paged_attn(self.q, self.planes[0], self.planes[1], c_table, self.nv, self.dense, self.ws3, lse=self.lse)

    eager, captured = Step(), Step()
    captured.load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # a first run outside the capture, undone by setting the counts back
        captured.run()
        captured.nv.copy_(ints(past))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.run()
    other = torch.cuda.Stream()
    for i in range(5):
        eager.load(i)
        captured.load(i)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            eager.run()
        torch.cuda.synchronize()
        for name in ("nv", "scores", "idx", "sparse", "dense", "lse"):
            assert torch.equal(getattr(eager, name), getattr(captured, name)), (i, name)
        for a, b in zip(eager.planes, captured.planes):
            assert torch.equal(a, b)
    assert csa2.csa2_get_last_error() == 0


# ---- refusals of the binding ------------------------------------------------------------------


def test_binding_refuses_shapes_types_and_strides(csa2):
    c = Cache(csa2, [20, 30], 16, 90)
    q = normal(gen(91), 2, 64, 512)
    out, ws = torch.empty_like(q), csa2.paged_attn_workspace(2, 2)
    good = dict(q=q, kv_data=c.kv_data, kv_scale=c.kv_scale, page_table=c.table, n_visible=c.n_visible, out=out, workspace=ws)
    csa2.csa2_paged_attn(**good)
    for change in (dict(q=q.float()), dict(q=q[:, :32].contiguous()), dict(q=q.transpose(0, 1)), dict(out=out[:1]),
                   dict(kv_data=c.kv_data[:-1]), dict(kv_scale=c.kv_scale[:, :, :16].contiguous()),
                   dict(page_table=c.table.long()), dict(page_table=c.table[:1]), dict(n_visible=c.n_visible.cpu()),
                   dict(cu_q=ints([0, 2])), dict(lse=torch.empty(2, 63, device="cuda"))):
        with pytest.raises(ValueError):
            csa2.csa2_paged_attn(**dict(good, **change))
    with pytest.raises(csa2.Csa2Error) as e:
        csa2.csa2_paged_attn(**dict(good, workspace=ws[:256]))
    assert e.value.status == -6
    odd = torch.zeros(4, 24, 256, dtype=torch.uint8, device="cuda"), torch.zeros(4, 24, 32, dtype=torch.uint8, device="cuda")
    with pytest.raises(csa2.Csa2Error) as e:
        csa2.csa2_paged_attn(**dict(good, kv_data=odd[0], kv_scale=odd[1]))
    assert e.value.status == -2
    x, rope = normal(gen(92), 4, 2, 64), angles(8, 32)
    for bad in ((x[0], rope, None, x[0]), (x, rope[..., 0].contiguous(), None, x), (x, rope.double(), None, x),
                (x, rope, ints([1, 2]), x), (x, rope, None, x[:2])):
        with pytest.raises(ValueError):
            csa2.csa2_rope(*bad)
    with pytest.raises(ValueError):
        csa2.csa2_paged_kv_append(x[0], x[0], *c.planes, c.table, c.n_visible)
