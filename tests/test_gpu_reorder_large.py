"""Pages of any power of two of entries are accepted: one that holds more than 2^31 bytes
of codes is copied whole when it is partly filled."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [(1 << 23) - 1, 1 << 23, (1 << 23) + 5])
def test_a_page_of_more_than_2_gib(fill):
    """2^31 bytes are 2^23 entries; one entry less, and the copy's last step passes them."""
    from fp4_kv_cache_02_gb300 import csa2
    page = 1 << 24
    g = torch.Generator(device="cuda").manual_seed(fill)
    planes = {}
    for name, width in (("kv_data", 256), ("kv_scale", 32), ("ik_data", 64), ("ik_scale", 4)):
        p = planes[name] = torch.full((2, page, width), 0x5A, dtype=torch.uint8, device="cuda")
        # (random words, repeated with a period that is no power of two)
        p[0].view(-1)[:fill * width].view(torch.int32).copy_(
            torch.randint(-2 ** 31, 2 ** 31, (1000003,), generator=g, device="cuda", dtype=torch.int32).repeat(fill * width // 4000012 + 1)[:fill * width // 4])
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table_out, n_out = ints(-1, -1).view(2, 1), ints(0, 0)
    before = {name: p[0].clone() for name, p in planes.items()}
    csa2.csa2_paged_reorder(ints(0, 0), ints(-1, 1), ints(0).view(1, 1), ints(fill), table_out, n_out, **planes)
    assert csa2.csa2_get_last_error() == 0
    assert table_out.view(-1).tolist() == [0, 1] and n_out.tolist() == [fill, fill]
    for name, p in planes.items():
        assert torch.equal(p[0], before[name]), name
        assert torch.equal(p[1, :fill], p[0, :fill]), name
        assert (p[1, fill:] == 0x5A).all(), name
