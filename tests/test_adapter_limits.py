"""The largest weights that the dropout and grouped layers take, refused on the
host beyond them."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def nf():
    import nf4_base_lora_b200 as nf
    return nf


def test_a_weight_of_almost_two_to_the_31_rows(nf):
    """Its steps of 64 rows are counted in 31 bits: (rows + 63) / 64 in the kernels."""
    top, P = 1 << 31, ctypes.c_void_p
    for rows, fits in ((top - 64, True), (top - 56, False), (top - 8, False)):
        for size in (nf.qlora_linear_dropout_fwd_workspace_bytes, nf.qlora_linear_dropout_bwd_workspace_bytes):
            assert (size(1, rows, 64, 8) > 0) == fits, rows
        assert (nf.qlora_grouped_fwd_workspace_bytes(1, 2, rows // 2 // 8 * 8, 64, 8) > 0) or not fits
        if fits:
            continue
        w = nf.Nf4TensorStruct(rows, 64, *(1 << k for k in (20, 21, 22, 23)))
        rc = nf.lib.qlora_linear_dropout_fwd(ctypes.byref(w), P(1 << 24), P(1 << 25), 8, 1.0, None, P(1 << 26), 1,
                                             P(1 << 27), None, P(1 << 28), 1 << 40, None)
        assert rc == -2 and b"rows" in nf.lib.nf4lora_last_error_string()


def test_sizes_that_overflow_64_bits(nf):
    big = (1 << 31) - 64
    assert nf.qlora_grouped_fwd_workspace_bytes(1, 4096, big, big, 8) == 0
    assert nf.qlora_grouped_bwd_workspace_bytes(1, 4096, big, big, 8) == 0
