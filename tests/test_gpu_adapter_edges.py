"""Edges of the dropout and grouped layers that their kernels treat apart, on the
GPU against 64-bit results."""
import pytest
import torch

from adapter_ref import check, reference
from test_gpu_dropout import rng_tensor
from test_gpu_grouped import make, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nf():
    import nf4_base_lora_b200 as nf
    return nf


def compare(nf, E, N, K, r, counts, p, dq=True, first=0, behind=0, s=0.5, state=(3, 9)):
    """Forward and backward against the 64-bit results; rows outside the groups
    hold NaN and keep what the outputs had."""
    off, offsets = offsets_of(counts, first)
    M = off[-1] + behind
    w, W, d = make(nf, E, N, K, r, M, dq)
    rng = rng_tensor(state) if p else None
    inside = slice(off[0], off[-1])
    X, dY = torch.full_like(d["X"], float("nan")), torch.full_like(d["dY"], float("nan"))
    X[inside], dY[inside] = d["X"][inside], d["dY"][inside]
    Y, T, dX = torch.full_like(dY, 3.0), torch.full((M, r), 3.0, device="cuda"), torch.full_like(X, 3.0)
    nf.qlora_grouped_fwd(w, d["A"], d["B"], s, X, offsets, p, rng, Y=Y, T=T)
    _, dA, dB = nf.qlora_grouped_bwd(w, d["A"], d["B"], s, X, T, dY, offsets, p, rng, dX=dX)
    torch.cuda.synchronize()
    nf.device_status()
    ref = reference(W, d["A"], d["B"], d["X"], d["dY"], off, s, p, state)
    for name, got in (("T", T), ("Y", Y), ("dX", dX)):
        check(got, ref, name, inside)
        assert (got[:off[0]] == 3.0).all() and (got[off[-1]:] == 3.0).all(), name
    check(dA, ref, "dA")
    check(dB, ref, "dB")


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("r", [8, 72])
def test_a_group_may_end_on_any_row_of_a_step(nf, p, r):
    """dA and dB contract over 64 rows a step; the rows behind a group's end are
    the next group's, and NaN behind the last one."""
    counts = [64 * (i % 4) + i for i in range(1, 64, 2)]
    compare(nf, len(counts), 72, 320, r, counts, p, first=2, behind=61)


def elapsed_ms(f):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    f()
    a.record()
    f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("E", [100, 4096])
def test_offsets_that_break_the_rule_ask_for_no_more_work(nf, E):
    """Offsets that jump between 0 and M clamp every other group to all rows;
    the call does no more than one division of the rows can need."""
    M = 1 << 16
    w, W, d = make(nf, E, 8, 64, 4, M)
    out = {"Y": torch.empty_like(d["dY"]), "T": torch.empty((M, 4), device="cuda")}
    good = torch.linspace(0, M, E + 1, device="cuda").to(torch.int32)
    bad = (torch.arange(E + 1, device="cuda") % 2 * M).to(torch.int32)
    ws = torch.empty(nf.qlora_grouped_bwd_workspace_bytes(M, E, 8, 64, 4), dtype=torch.uint8, device="cuda")

    def call(offsets):
        nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets, workspace=ws, **out)
        nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], out["T"], d["dY"], offsets, workspace=ws)
    t_good = elapsed_ms(lambda: call(good))
    nf.device_status()
    t_bad = elapsed_ms(lambda: call(bad))
    with pytest.raises(nf.Nf4Error, match="offsets"):
        nf.device_status()
    # E / 2 times the rows if every group were run
    assert t_bad <= 8 * t_good + 1.0, (t_bad, t_good)


# none of these leaves a group a row, or only the last one
NO_ROWS = ([64, 40, 20, 0], [-1] * 4, [65] * 4, [64, 64, 64, 65], [-5, -3, -1, 0], [1 << 30] * 4)


@pytest.mark.parametrize("off", [*NO_ROWS, [0, 40, 20, 64]], ids=str)
def test_every_call_reports_offsets_that_break_the_rule(nf, off):
    """Whatever the call asks for, and also where the clamped groups have no rows
    so that no kernel has work."""
    E, N, K, r, M = 3, 128, 128, 8, 64
    w, W, d = make(nf, E, N, K, r, M)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    T = torch.zeros((M, r), device="cuda")

    def reported(f):
        f()
        with pytest.raises(nf.Nf4Error, match="offsets"):
            nf.device_status()
        nf.device_status()
    reported(lambda: nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets))
    for dx, da, db in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 0, 1)):
        for saved in (T, None):
            reported(lambda: nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], saved, d["dY"], offsets,
                                                  need_dx=bool(dx), need_da=bool(da), need_db=bool(db)))
