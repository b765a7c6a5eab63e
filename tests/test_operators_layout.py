"""CPU check: the binding's own count of a laid-out matrix's bytes is the library's."""

import pytest


@pytest.mark.parametrize("form", ["e8m0", "e4m3"])
def test_the_bindings_count_of_a_matrix(form):
    from fp4_kv_cache_02_gb300 import csa2
    kind = csa2.FP4_FORMATS[form]
    assert sorted(csa2.FP4_FORMATS.values()) == list(range(len(csa2._BLOCK_BYTES)))
    for n_out in (0, 1, 127, 128, 129, 640, 4096, 128259, 1 << 22):
        for n_in in (32, 224, 256, 288, 4096, 32768, 1 << 20):
            assert csa2._weights_bytes(n_out, n_in, kind) == csa2.csa2_fp4_weights_size(n_out, n_in, form), (n_out, n_in)
