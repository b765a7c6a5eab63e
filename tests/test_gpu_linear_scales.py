"""E8M0 scales over their whole range, on both sides of 64 tokens: the weights are
exact, 6 x 2^127 and 1/2 x 2^-127 among them, and only a result that is too large for
fp32 is infinite.

The bound is that of test_gpu_linear.py. Where sums are subnormal in fp32 each
rounding is off by up to 2^-150 instead; the larger form of the product holds a
quarter of its sums and rounds twice every 16 inputs, the other half of them, in eight
columns, twice every 64, and at most 40 operations follow: (n_in / 4 + 40) 2^-148.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

TOKENS = [1, 3, 20, 64, 65, 90, 300]


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_02_gb300 import csa2 as m
    return m


def values(data, scale):
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    v = torch.cat([v, -v])
    w = torch.stack([v[(data & 15).long()], v[(data >> 4).long()]], -1).flatten(-2)
    powers = torch.tensor([2.0 ** (e - 127) for e in range(256)], dtype=torch.float64, device="cuda")  # (ldexp's are fp32 ones)
    return w * powers[scale.long()].repeat_interleave(32, -1)


def call(csa2, x, data, scale, factor=1.0):
    out, out32 = torch.empty(x.shape[0], data.shape[0], dtype=torch.bfloat16, device="cuda"), torch.empty(x.shape[0], data.shape[0], device="cuda")
    csa2.csa2_fp4_linear(x, csa2.fp4_weights(data, scale, "e8m0"), out, csa2.fp4_linear_workspace(x.shape[0], x.shape[1], "e8m0"), "e8m0",
                         scale=factor, out_f32=out32)
    assert csa2.csa2_get_last_error() == 0
    assert torch.allclose(out, out32.bfloat16(), rtol=0.0, atol=0.0, equal_nan=True)
    return out32


@pytest.mark.parametrize("T", TOKENS)
def test_every_value_of_every_scale(csa2, T):
    """One channel of each token is a power of two, so that outputs are the weights' values themselves: 255 scales x 16 codes."""
    n_in = 64
    code = torch.arange(16, dtype=torch.uint8, device="cuda").repeat(255)
    data = (code * 17)[:, None].repeat(1, n_in // 2)
    scale = torch.arange(255, dtype=torch.uint8, device="cuda").repeat_interleave(16)[:, None].repeat(1, n_in // 32)
    x = torch.zeros(T, n_in, device="cuda")
    at = torch.arange(T, device="cuda") * 7 % n_in
    power = torch.arange(T, device="cuda") % 5 - 9
    x[torch.arange(T, device="cuda"), at] = torch.exp2(power.float())
    ref = x.double() @ values(data, scale).T
    assert torch.equal(ref.float().double(), ref) and ref.abs().max() >= 2.0 ** 120  # (a multiple of 2^-137: exact in fp32)
    assert torch.equal(call(csa2, x.bfloat16(), data, scale).double(), ref)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("n_in", [256, 2080])
@pytest.mark.parametrize("codes", [(252, 252), (253, 253), (254, 254), (250, 254), (0, 3), (0, 254)])
def test_scales_at_both_ends(csa2, T, n_in, codes):
    g = torch.Generator(device="cuda").manual_seed(T + n_in + codes[0])
    n_out = 150
    x = (torch.randn(T, n_in, generator=g, device="cuda").clamp(-4, 4) * 2.0 ** -16).bfloat16()  # (2,080 x 6 x 2^127 x 2^-14 < 2^128)
    data = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(codes[0], codes[1] + 1, (n_out, n_in // 32), generator=g, device="cuda").to(torch.uint8)
    out32 = call(csa2, x, data, scale, 0.5)
    xd, w = x.double(), values(data, scale)
    A = xd.abs() @ w.abs().T
    M = xd.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1) @ w.abs().T
    bound = 2.0 ** -22 * M + (n_in / 64 + 20) * 2.0 ** -22 * (4 * A + 2.0 ** -20 * M) + (n_in / 4 + 40) * 2.0 ** -148
    assert out32.isfinite().all()
    assert (out32.double() - 0.5 * (xd @ w.T)).abs().le(0.5 * bound + 2.0 ** -149).all()


@pytest.mark.parametrize("T", TOKENS)
def test_results_past_fp32_and_scales_that_are_nan(csa2, T):
    n_in = 128
    x = torch.full((T, n_in), 2.0, device="cuda").bfloat16()
    data = torch.full((4, n_in // 2), 0x77, dtype=torch.uint8, device="cuda")  # sixes
    scale = torch.full((4, n_in // 32), 127, dtype=torch.uint8, device="cuda")
    scale[1] = 254
    scale[2, 1] = 255
    data[3] = 0xFF  # less six
    scale[3] = 254
    out = call(csa2, x, data, scale)
    assert (out[:, 0] == 12.0 * n_in).all() and out[:, 2].isnan().all()
    assert (out[:, 1] == float("inf")).all() and (out[:, 3] == -float("inf")).all()
