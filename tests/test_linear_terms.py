"""Up to 64 tokens a row enters the products with 4-bit weights as eight vectors, the
base-8 digits of its channels on a grid 2^-22 of their block's largest power of two
apart. The header promises exactness for channels within 2^-14 of their block's
largest; here every one of the eight has to be right for it.

A block holds one large channel, whose weights are 0, and one channel of eight
significant bits 2^-j of it, whose weight is 1, 2 or -1; the others are 0. j is the
same for all of a token's blocks, 0 .. 14. A small channel is a multiple of 2^(14 - j) of
the grid's units, so of the place of the digit that holds this bit, 2^(12 - j) at least, and
its digits add up to less than 2^(23 - j). So all sums of digits, over up to 256 blocks and
with weights of up to 2, are multiples of 2^(12 - j) below 2^(32 - j): 20 bits, which
every fp32 sum holds exactly. The outputs have to be equal, in every form of the product.
"""

import numpy as np
import pytest
import torch

PER = {"e8m0": 32, "e4m3": 16}
# terms made by the product, in one CTA and in clusters; ahead, in clusters and single CTAs; runs; two tiles of tokens; and
# the tokens' own values
SHAPES = [(1, 256, 40), (1, 4096, 640), (2, 2048, 300), (3, 1024, 520), (8, 2048, 700), (12, 512, 6000), (9, 96, 40000),
          (20, 288, 20000), (32, 1024, 200), (64, 1056, 300), (90, 1024, 300)]


def rows_of_two(g, T, n_in, per, j):
    """(x in 64 bits, places of the large channels, of the small ones): small ones 2^-j of the large, j by token."""
    blocks = n_in // per
    sign = lambda *s: 1.0 - 2.0 * torch.randint(0, 2, s, generator=g, dtype=torch.float64)
    x = torch.zeros(T, blocks, per, dtype=torch.float64)
    block = torch.arange(blocks)
    large = torch.randint(0, per, (blocks,), generator=g)
    small = (large + torch.randint(1, per, (blocks,), generator=g)) % per
    m = 2 * torch.randint(64, 128, (T, blocks), generator=g) + 1  # odd, eight bits
    power = torch.randint(-40, 41, (T, 1), generator=g).double()
    x[:, block, large] = sign(T, blocks) * torch.exp2(power)
    x[:, block, small] = sign(T, blocks) * m.double() * torch.exp2(power - 7 - j[:, None].double())
    return x.view(T, n_in), block * per + large, block * per + small


def matrix(g, n_out, n_in, per, small):
    """Codes [n_out][n_in / 2] of weights that are 1, 2 or -1 for the small channels and 0 for all others."""
    codes = torch.zeros(n_out, n_in, dtype=torch.uint8)
    codes[:, small] = torch.tensor([2, 4, 10], dtype=torch.uint8)[torch.randint(0, 3, (n_out, len(small)), generator=g)]
    weight = torch.zeros(n_out, n_in, dtype=torch.float64)
    weight[codes == 2], weight[codes == 4], weight[codes == 10] = 1.0, 2.0, -1.0
    return codes[:, 0::2] | codes[:, 1::2] << 4, weight


def digits(x, per, left_out=()):
    """The value of rows x as the sum of their eight digits, by the definition, without those named."""
    b = x.view(x.shape[0], -1, per).numpy()
    e = np.frexp(np.abs(b).max(-1, keepdims=True))[1] - 1
    n = np.rint(np.ldexp(b, 21 - e)).astype(np.int64)  # multiples of 2^(e - 21), below 2^22
    total = np.zeros(b.shape)
    for d in range(8):  # from the last: -4 .. 3
        digit = ((n + 4) & 7) - 4
        n = (n - digit) >> 3
        if 7 - d not in left_out:
            total += np.ldexp(digit.astype(np.float64), 3 * d + e - 21)
    assert (n == 0).all()
    return torch.from_numpy(total).view(x.shape)


def places(T, turn):
    """The small channels' distance 2^-j by token: all of 0 .. 14 between the turns."""
    return (torch.arange(T) * 4 + turn) % 15


@pytest.mark.parametrize("form", PER)
def test_the_rows_need_every_digit(form):
    """On the CPU: the digits give the rows exactly, and without any one of them the outputs differ."""
    for T, n_in, n_out in [(1, 256, 40), (3, 1024, 50), (20, 288, 30)]:
        wrong = set()
        for turn in range(15):
            g = torch.Generator().manual_seed(100 * turn + T)
            x, large, small = rows_of_two(g, T, n_in, PER[form], places(T, turn))
            _, w = matrix(g, n_out, n_in, PER[form], small)
            assert torch.equal(x.bfloat16().double(), x)
            assert torch.equal(digits(x, PER[form]), x)
            ref = x @ w.T
            assert torch.equal(ref.float().double(), ref)
            wrong |= {d for d in range(8) if not torch.equal(digits(x, PER[form], (d,)) @ w.T, ref)}
        assert wrong == set(range(8))


@pytest.mark.gpu
@pytest.mark.parametrize("form", PER)
@pytest.mark.parametrize("shape", SHAPES)
def test_channels_within_their_reach_are_exact(shape, form):
    from fp4_kv_cache_02_gb300 import csa2
    T, n_in, n_out = shape
    for turn in range(15) if T < 15 else range(0, 15, 5):
        g = torch.Generator().manual_seed(100 * turn + T)
        x, large, small = rows_of_two(g, T, n_in, PER[form], places(T, turn))
        data, w = matrix(g, n_out, n_in, PER[form], small)
        one = 127 if form == "e8m0" else 0x38
        scale = torch.full((n_out, n_in // PER[form]), one, dtype=torch.uint8, device="cuda")
        out32 = torch.full((T, n_out), 7.0, device="cuda")
        csa2.csa2_fp4_linear(x.bfloat16().cuda(), csa2.fp4_weights(data.cuda(), scale, form), None,
                             csa2.fp4_linear_workspace(T, n_in, form), form, out_f32=out32)
        ref = x.cuda() @ w.T.cuda()
        assert torch.equal(out32.double(), ref), (turn, (out32.double() - ref).abs().max())
    assert csa2.csa2_get_last_error() == 0
