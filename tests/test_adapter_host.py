"""Refusals of the adapter-dropout and grouped-expert entry points, all on the
host before a device is touched, and the sizes they report."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def nf():
    import nf4_base_lora_b200 as nf
    return nf


P = ctypes.c_void_p
INVALID, SHAPE, ALIGN, WORK, CUDA = -1, -2, -3, -4, -5
A, B, X, Y, WS, OFF, G, ST = (P(1 << k) for k in (24, 25, 26, 27, 28, 29, 30, 31))
BIG = 1 << 40


def weight(nf, d_out=256, d_in=128):
    s = nf.Nf4TensorStruct()
    assert nf.lib.nf4_tensor_from_buffer(ctypes.byref(s), P(1 << 20), nf.nf4_packed_bytes(d_out, d_in), d_out,
                                         d_in) == 0
    return s


def drop(nf, p, state=1 << 31):
    return ctypes.byref(nf.LoraDropoutStruct(p, state))


def test_dropout_refusals(nf):
    f = nf.lib.lora_dropout
    assert f(X, -1, 0, drop(nf, 0.1), Y, None) == INVALID
    assert f(X, 8, 2, drop(nf, 0.1), Y, None) == INVALID          # unknown type
    assert f(X, 8, 0, None, Y, None) == INVALID
    for p in (-0.1, 1.0, float("nan"), float("inf"), 1 - 2.0 ** -17):
        assert f(X, 8, 0, drop(nf, p), Y, None) == INVALID, p
    assert b"nothing would be kept" in nf.lib.nf4lora_last_error_string()
    assert f(X, 8, 0, drop(nf, 0.1, None), Y, None) == INVALID    # no state
    assert f(X, 8, 0, drop(nf, 0.1, (1 << 31) + 4), Y, None) == ALIGN
    assert f(None, 8, 0, drop(nf, 0.1), Y, None) == INVALID
    assert f(P((1 << 26) + 2), 8, 0, drop(nf, 0.1), Y, None) == ALIGN
    assert f(None, 0, 0, drop(nf, 0.1), None, None) == 0          # nothing to do
    assert f(X, 8, 1, drop(nf, 0.1), Y, None) == CUDA             # passes the checks, no device here


def fwd(nf, w, d=None, x=X, m=16, y=Y, t=None, ws=WS, n=BIG, r=8, s=2.0):
    return nf.lib.qlora_linear_dropout_fwd(ctypes.byref(w), A, B, r, s, d, x, m, y, t, ws, n, None)


def gfwd(nf, w, e=2, d=None, x=X, m=16, off=OFF, y=Y, t=None, ws=WS, n=BIG, r=8, s=2.0):
    return nf.lib.qlora_grouped_fwd(ctypes.byref(w), e, A, B, r, s, d, x, m, off, y, t, ws, n, None)


def gbwd(nf, w, e=2, d=None, x=X, t=None, dy=Y, m=16, off=OFF, dx=None, da=G, db=None, acc=0, ws=WS, n=BIG, r=8):
    return nf.lib.qlora_grouped_bwd(ctypes.byref(w), e, A, B, r, 2.0, d, x, t, dy, m, off, dx, da, db, acc, ws, n,
                                    None)


def test_layer_refusals(nf):
    w = weight(nf)
    assert fwd(nf, w) == CUDA
    assert fwd(nf, w, drop(nf, 0.1)) == CUDA
    assert fwd(nf, w, drop(nf, 1.0)) == INVALID
    assert fwd(nf, w, drop(nf, 0.1, None)) == INVALID
    assert fwd(nf, w, drop(nf, 0.0, None)) == CUDA                # p = 0 needs no state
    assert fwd(nf, w, r=0) == INVALID and fwd(nf, w, r=257) == INVALID
    assert fwd(nf, w, s=float("inf")) == INVALID
    assert fwd(nf, w, x=None) == INVALID and fwd(nf, w, y=None) == INVALID
    assert fwd(nf, w, m=-1) == INVALID and fwd(nf, w, m=1 << 31) == INVALID
    assert fwd(nf, w, x=P((1 << 26) + 8)) == ALIGN and fwd(nf, w, t=P((1 << 26) + 8)) == ALIGN
    need = nf.qlora_linear_dropout_fwd_workspace_bytes(16, 256, 128, 8)
    assert fwd(nf, w, n=need - 1) == WORK and fwd(nf, w, ws=None) == WORK
    assert fwd(nf, w, ws=P((1 << 28) + 16)) == ALIGN
    assert fwd(nf, w, m=0, x=None, y=None, ws=None) == 0


def test_grouped_refusals(nf):
    w = weight(nf)
    assert gfwd(nf, w) == CUDA
    for e in (0, -1, nf.lib and 4097):
        assert gfwd(nf, w, e=e) == INVALID
    assert gfwd(nf, w, e=3) == SHAPE                              # 256 rows, 3 experts
    assert gfwd(nf, w, e=64) == SHAPE                             # 4 rows each: not a multiple of 8
    assert gfwd(nf, w, off=None) == INVALID
    assert gfwd(nf, w, off=P((1 << 29) + 2)) == ALIGN
    assert gfwd(nf, w, m=0, x=None, y=None, off=None, ws=None) == 0
    need = nf.qlora_grouped_fwd_workspace_bytes(16, 2, 128, 128, 8)
    assert gfwd(nf, w, n=need - 1) == WORK


def test_backward_refusals(nf):
    w = weight(nf)
    assert gbwd(nf, w) == CUDA
    assert gbwd(nf, w, dy=None) == INVALID
    assert gbwd(nf, w, acc=2) == INVALID
    assert gbwd(nf, w, x=None) == INVALID                         # dA needs X
    assert gbwd(nf, w, x=None, da=None, db=G) == INVALID          # dB without T needs X
    assert gbwd(nf, w, x=None, t=P(1 << 33), da=None, db=G) == CUDA
    assert gbwd(nf, w, x=None, da=None, dx=G) == CUDA             # dX alone
    assert gbwd(nf, w, da=P((1 << 30) + 4)) == ALIGN
    assert gbwd(nf, w, da=None) == 0                              # nothing asked for
    assert gbwd(nf, w, m=0, acc=1, dy=None, off=None, ws=None) == 0
    need = nf.qlora_grouped_bwd_workspace_bytes(16, 2, 128, 128, 8)
    assert gbwd(nf, w, n=need - 1) == WORK


def test_sizes(nf):
    g = nf.qlora_grouped_bwd_workspace_bytes
    assert nf.qlora_grouped_fwd_workspace_bytes(0, 2, 128, 128, 8) == 0
    assert g(16, 0, 128, 128, 8) == 0 and g(16, 2, 128, 100, 8) == 0 and g(16, 2, 128, 128, 300) == 0
    assert 0 < g(16, 8, 4096, 4096, 16) < g(4096, 8, 4096, 4096, 16)
    # an odd rank pads B: E * d_out rows of 8 elements more
    assert g(16, 8, 4096, 4096, 15) >= g(16, 8, 4096, 4096, 16) + 8 * 4096 * 16 * 2
    assert nf.qlora_linear_dropout_bwd_workspace_bytes(100, 512, 256, 8) == g(100, 1, 512, 256, 8)


def test_binding_refuses_tensors_of_the_wrong_kind(nf):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nf.lora_dropout(x, 0.1, None)                             # not on a GPU
    with pytest.raises(ValueError):
        nf.lora_dropout(x.half(), 0.1, None)


def test_a_weight_of_too_many_blocks_is_refused(nf):
    w = weight(nf, 1 << 23, 1 << 15)                              # 2^32 blocks of 64
    assert fwd(nf, w) == SHAPE and gfwd(nf, w) == SHAPE and gbwd(nf, w) == SHAPE
    assert nf.qlora_grouped_fwd_workspace_bytes(16, 2, 1 << 22, 1 << 15, 8) == 0
    w = weight(nf, (1 << 23) - 16, 1 << 15)
    assert fwd(nf, w) == CUDA and gfwd(nf, w) == CUDA             # passes the checks, no device here
    assert nf.qlora_grouped_fwd_workspace_bytes(16, 2, (1 << 22) - 8, 1 << 15, 8) > 0
