"""lora_dropout in place, beside its input, and where it would overwrite elements
that it has still to read (host checks only)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def nf():
    import nf4_base_lora_b200 as nf
    return nf


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("dtype,size", [(0, 2), (1, 4)])
def test_a_partial_overlap_is_refused(nf, p, dtype, size):
    base, n = 1 << 26, 4096
    drop = ctypes.byref(nf.LoraDropoutStruct(p, 1 << 31))

    def call(x, out):
        return nf.lib.lora_dropout(ctypes.c_void_p(x), n, dtype, drop, ctypes.c_void_p(out), None)
    no_device = -5                       # passes the checks, no device here
    assert call(base, base) == no_device
    assert call(base, base + n * size) == no_device and call(base + n * size, base) == no_device
    for off in (16, n * size // 2, n * size - 16):
        assert call(base, base + off) == -1 and call(base + off, base) == -1
    assert b"overlaps" in nf.lib.nf4lora_last_error_string()
