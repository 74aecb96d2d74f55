"""Edges of the dropout and grouped layers that their kernels treat apart, on the
GPU against 64-bit results."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

from adapter_ref import check, reference
from group_cases import CASES
from test_gpu_dropout import rng_tensor
from test_gpu_grouped import make, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nf():
    import nf4_base_lora_b200 as nf
    return nf


def compare(nf, E, N, K, r, counts, p, dq=True, first=0, behind=0, s=0.5, state=(3, 9)):
    """Forward and backward against the 64-bit results; rows outside the groups
    hold NaN and keep what the outputs had.  E None: the dense layer."""
    dense, E = E is None, E or 1
    off, offsets = offsets_of(counts, first)
    M = off[-1] + behind
    w, W, d = make(nf, E, N, K, r, M, dq)
    rng = rng_tensor(state) if p else None
    inside = slice(off[0], off[-1])
    X, dY = torch.full_like(d["X"], float("nan")), torch.full_like(d["dY"], float("nan"))
    X[inside], dY[inside] = d["X"][inside], d["dY"][inside]
    Y, T, dX = torch.full_like(dY, 3.0), torch.full((M, r), 3.0, device="cuda"), torch.full_like(X, 3.0)
    if dense:
        a, b = d["A"][0], d["B"][0]
        nf.qlora_linear_dropout_fwd(w, a, b, s, X, p, rng, Y=Y, T=T)
        _, dA, dB = nf.qlora_linear_dropout_bwd(w, a, b, s, X, T, dY, p, rng, dX=dX)
        dA, dB = dA[None], dB[None]
    else:
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


@pytest.mark.parametrize("p,dq", [(0.0, False), (0.2, True)])
@pytest.mark.parametrize("name", CASES)
def test_pairs_that_walk_several_tiles_and_split_contractions(nf, name, p, dq):
    E, N, K, r, rows = CASES[name][:5]
    compare(nf, E, N, K, r, rows, p, dq)


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


def signed(g, rows, cols):
    """|normal| with one sign a column, so that sums over rows of infinities have one."""
    sign = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    return ((torch.randn(rows, cols, generator=g, device="cuda").abs() + 0.01) * sign).bfloat16()


def layer_calls(nf, kind, w, A, B, s, X, dY, T=None):
    """(Y, T, dX, dA, dB) of the plain, the dropout (p = 0) or the grouped layer;
    T: what the backward gets, else the forward's."""
    if kind == "plain":
        Y, T0 = nf.qlora_linear_fwd(w, A, B, s, X)
        return (Y, T0, *nf.qlora_linear_bwd(w, A, B, s, X, T0 if T is None else T, dY))
    if kind == "dropout":
        Y, T0 = nf.qlora_linear_dropout_fwd(w, A, B, s, X, 0.0, None)
        return (Y, T0, *nf.qlora_linear_dropout_bwd(w, A, B, s, X, T0 if T is None else T, dY, 0.0, None))
    offsets = torch.tensor([0, X.shape[0]], dtype=torch.int32, device="cuda")
    Y, T0 = nf.qlora_grouped_fwd(w, A[None], B[None], s, X, offsets)
    dX, dA, dB = nf.qlora_grouped_bwd(w, A[None], B[None], s, X, T0 if T is None else T, dY, offsets)
    return Y, T0, dX, dA[0], dB[0]


def same_or_close(got, ref, name):
    """NaN and infinities exactly; finite elements to 2^-6 of the largest (a rounding is 2^-8)."""
    got, fin = got.double(), torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), name
    assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)]), name
    assert ((got - ref).abs()[fin] <= 2.0 ** -6 * ref.abs()[fin].max()).all() if fin.any() else True, name


@pytest.mark.parametrize("M", [1, 5, 200])
@pytest.mark.parametrize("kind", ["plain", "dropout", "grouped"])
def test_an_infinite_t_or_v_gives_the_formulas_infinities(nf, kind, M):
    """T and V enter the products as pairs of 16-bit values; an infinite one, from
    an infinite element of A or B, is the formula's signed infinity in all that
    follows from it, never a NaN."""
    N, K, r, s = 136, 192, 8, 0.5
    g = torch.Generator(device="cuda").manual_seed(M)
    w = nf.nf4_quantize(torch.randn(N, K, generator=g, device="cuda") * 0.02)
    W = nf.nf4_dequantize(w).double()
    X, dY = signed(g, M, K), signed(g, M, N)
    A, B = signed(g, K, r).t().contiguous(), signed(g, N, r)
    for which in "AB":
        a, b = A.clone(), B.clone()
        (a if which == "A" else b)[(3, 70) if which == "A" else (70, 3)] = float("inf")
        Y, T, dX, dA, dB = layer_calls(nf, kind, w, a, b, s, X, dY)
        x, dy, ad, bd = X.double(), dY.double(), a.double(), b.double()
        if which == "A":
            t = s * (x @ ad.T)
            same_or_close(T, t, "T")
            same_or_close(Y, x @ W.T + t @ bd.T, "Y")
            same_or_close(dB, dy.T @ t, "dB")
        else:
            v = s * (dy @ bd)
            same_or_close(dX, dy @ W + v @ ad, "dX")
            same_or_close(dA, v.T @ x, "dA")
        torch.cuda.synchronize()
    nf.device_status()


@pytest.mark.parametrize("M", [1, 5, 200])
@pytest.mark.parametrize("kind", ["plain", "dropout", "grouped"])
def test_a_t_or_v_beyond_the_16_bit_range_is_exact(nf, kind, M):
    """2^128 - 2^118 is a finite fp32 value that rounds to infinity in 16 bits.
    Its products with factors of about 2^-100 are finite: within the roundings
    (2^-8 of the result and what the pair leaves, 2^-16)."""
    N, K, r = 136, 192, 8
    big, tiny = 2.0 ** 127, 2.0 ** -100
    g = torch.Generator(device="cuda").manual_seed(7)
    w = nf.nf4_quantize(torch.zeros(N, K, device="cuda"))
    X, dY = torch.zeros(M, K, device="cuda"), torch.zeros(M, N, device="cuda")
    A, B = torch.full((r, K), tiny, device="cuda"), torch.full((N, r), tiny, device="cuda")
    # T[:, 3] = V[:, 3] = 255 / 128 2^127 + 1.5 2^119
    for act, fac in ((X, A[3]), (dY, B[:, 3])):
        act[:, 0], act[:, 1] = 255 / 128, 1.5
        fac[0], fac[1] = big, 2.0 ** 119
    Y, T, dX, dA, dB = layer_calls(nf, kind, w, *(t.bfloat16() for t in (A, B)), 1.0, X.bfloat16(), dY.bfloat16())
    x, dy, a, b = X.double(), dY.double(), A.double(), B.double()
    t, v = x @ a.T, dy @ b
    assert torch.equal(T.double(), t.float().double()) and float(t[0, 3]) == 2.0 ** 128 - 2.0 ** 118
    for name, got, ref in (("Y", Y, t @ b.T), ("dX", dX, v @ a), ("dA", dA, v.T @ x), ("dB", dB, dy.T @ t)):
        # columns and rows that meet the large elements twice are infinite in 32 bits already
        fin = ref.abs() < 2.0 ** 120
        assert fin.any() and ((got.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -14) * ref.abs())[fin].all(), name


@pytest.mark.parametrize("which", ["dB", "dA"])
def test_gradients_over_many_rows_keep_their_precision(nf, which):
    """Tensor-core additions truncate, so a long sum of one sign is too small by up
    to a unit (2^-23) of the running sum an addition, half a unit on average, of a
    running sum that is half the result on average.  A row of 64 takes 8 additions
    (two halves of the pair, 16 rows each) and an accumulator 128 rows of 64 at
    most: 1024 2^-25 on average, however many rows there are.  To see more of the
    sum than the 8 bits of a gradient, it is accumulated onto the negative result
    rounded to them, which the kernels do in 32 bits: what comes out is at most 2^-8
    of the result, and rounded to 2^-8 of that."""
    M, r, wide, narrow = 1 << 18, 8, 11008, 64
    N, K = (wide, narrow) if which == "dB" else (narrow, wide)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = nf.nf4_quantize(torch.randn(N, K, generator=g, device="cuda") * 0.02)
    pos = lambda *s: torch.rand(s, generator=g, device="cuda") + 0.5
    A, B = pos(r, K).bfloat16(), pos(N, r).bfloat16()
    act = torch.empty((M, wide), dtype=torch.bfloat16, device="cuda")
    for i in range(0, M, 1 << 14):
        act[i:i + (1 << 14)] = pos(1 << 14, wide)
    other = pos(M, narrow).bfloat16()
    X, dY = (other, act) if which == "dB" else (act, other)
    T = pos(M, r)
    f = T if which == "dB" else dY.double() @ B.double()
    ref = torch.zeros((r, wide), dtype=torch.float64, device="cuda")
    for i in range(0, M, 1 << 14):
        ref += f[i:i + (1 << 14)].double().T @ act[i:i + (1 << 14)].double()
    grad = -(ref.t() if which == "dB" else ref).bfloat16().contiguous()
    before = grad.double()
    out = {"dA": grad} if which == "dA" else {"dB": grad}
    nf.qlora_linear_dropout_bwd(w, A, B, 1.0, X, T, dY, 0.0, None, need_dx=False, need_da=which == "dA",
                                need_db=which == "dB", accumulate=True, **out)
    got = grad.double() - before
    mean = (((got.t() if which == "dB" else got) - ref) / ref).mean()
    assert abs(float(mean)) <= 1024 * 2.0 ** -25 + 2.0 ** -16, float(mean)


@pytest.mark.parametrize("dq,N,K", [(True, 256, 256), (True, 64, 2048), (False, 24, 192)])
def test_an_expert_as_a_tensor_of_its_own(nf, dq, N, K):
    """The pointers that the header gives for one expert of a stack: merged with its
    adapter it is its weight plus s B A, rounded once to fp32 (64-bit sums)."""
    E, r, s = 3, 5, 0.75
    w, W, d = make(nf, E, N, K, r, 1, dq)
    full = w.struct
    for e in range(E):
        n = e * N * K
        one = nf.Nf4TensorStruct(N, K, full.codes + n // 2)
        if dq:
            one.qscale, one.scale2 = full.qscale + n // 64, full.scale2 + 4 * (n // 16384)
            one.scale_mean = full.scale_mean
        else:
            one.absmax = full.absmax + 4 * (n // 64)
        out = torch.empty((N, K), device="cuda")
        A, B = d["A"][e], d["B"][e]
        assert nf.lib.nf4_merge_lora(ctypes.byref(one), A.data_ptr(), B.data_ptr(), r, s, out.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream) == 0
        ref = W[e].double() + s * (B.double() @ A.double())
        assert ((out.double() - ref).abs() <= 2.0 ** -24 * ref.abs() * 1.001 + 1e-15).all()


@pytest.mark.parametrize("M", [5, 90, 700])
def test_layers_of_every_kind_in_one_chain(nf, M):
    """The kernels of all layers are programmatic dependents of one another.  Plain,
    dropout and grouped layers in turn, forward and backward in one workspace, each
    on what the one before wrote: synchronised after every call, back to back and
    replayed from a graph, the same bits."""
    D, r, E, p, s = 512, 16, 4, 0.1, 0.5
    w, W, d = make(nf, 1, D, D, r, M)
    we, _, de = make(nf, E, D, D, r, M, seed=1)
    A, B = d["A"][0], d["B"][0]
    rng = rng_tensor((4, 4))
    _, offsets = offsets_of([M // 3, 0, M - M // 3, 0])
    need = max(nf.qlora_fwd_workspace_bytes(M, D, D, r), nf.qlora_bwd_workspace_bytes(M, D, D, r),
               nf.qlora_grouped_fwd_workspace_bytes(M, E, D, D, r), nf.qlora_grouped_bwd_workspace_bytes(M, E, D, D, r),
               nf.qlora_linear_dropout_fwd_workspace_bytes(M, D, D, r),
               nf.qlora_linear_dropout_bwd_workspace_bytes(M, D, D, r))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    h = [d["X"]] + [new(M, D) for _ in range(6)]
    g = [d["dY"]] + [new(M, D) for _ in range(6)]
    t = [torch.empty((M, r), device="cuda") for _ in range(6)]
    dA = [new(E, r, D) if i % 3 == 2 else new(r, D) for i in range(6)]
    dB = [new(E, D, r) if i % 3 == 2 else new(D, r) for i in range(6)]

    def chain(after):
        for i in range(6):
            if i % 3 == 0:
                nf.qlora_linear_fwd(w, A, B, s, h[i], Y=h[i + 1], T=t[i], workspace=ws)
            elif i % 3 == 1:
                nf.qlora_linear_dropout_fwd(w, A, B, s, h[i], p, rng, Y=h[i + 1], T=t[i], workspace=ws)
            else:
                nf.qlora_grouped_fwd(we, de["A"], de["B"], s, h[i], offsets, p, rng, Y=h[i + 1], T=t[i], workspace=ws)
            after()
        for k, i in enumerate(reversed(range(6))):
            out = dict(dX=g[k + 1], dA=dA[i], dB=dB[i], workspace=ws)
            if i % 3 == 0:
                nf.qlora_linear_bwd(w, A, B, s, h[i], t[i], g[k], **out)
            elif i % 3 == 1:
                nf.qlora_linear_dropout_bwd(w, A, B, s, h[i], t[i], g[k], p, rng, **out)
            else:
                nf.qlora_grouped_bwd(we, de["A"], de["B"], s, h[i], t[i], g[k], offsets, p, rng, **out)
            after()
    everything = [*h[1:], *g[1:], *t, *dA, *dB]
    chain(torch.cuda.synchronize)
    first = [v.clone() for v in everything]
    assert all(torch.isfinite(v).all() for v in first)

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(everything, first))
        for v in everything:
            v.fill_(7.0)
    same()
    for _ in range(5):
        chain(lambda: None)
        same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
        chain(lambda: None)
    for _ in range(5):
        graph.replay()
        same()
    nf.device_status()


FIRST_CALL = """
import torch, sys
sys.path[:0] = ["tests"]
import nf4_base_lora_b200 as nf
from test_gpu_grouped import make, offsets_of
w, W, d = make(nf, 2, 256, 192, 12, 40)
off, offsets = offsets_of([30, 10])
rng = torch.tensor([1, 2], device="cuda")
def step():
    x = nf.lora_dropout(d["X"], 0.2, rng)
    y, t = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, x, offsets, 0.2, rng)
    return y, t, *nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, x, t, d["dY"], offsets, 0.2, rng)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
eager = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, eager))
nf.device_status()
print("same")
"""


def test_the_first_call_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "same" in out.stdout, out.stderr[-3000:]


def test_two_host_threads_at_once(nf):
    """Each thread its own stream, data and workspaces; the same bits as alone."""
    sets = [make(nf, 3, 256, 320, 16, 150, seed=i) for i in range(2)]
    _, offsets = offsets_of([70, 0, 80])
    rng = rng_tensor((5, 5))

    def step(w, d):
        y, t = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets, 0.1, rng)
        return (nf.lora_dropout(d["X"], 0.1, rng), y, t,
                *nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], t, d["dY"], offsets, 0.1, rng))
    alone = [step(w, d) for w, _, d in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = step(sets[i][0], sets[i][2])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong
    nf.device_status()
