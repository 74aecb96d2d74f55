"""The layer of a mixture of experts on the GPU against 64-bit results: ragged
groups, empty experts, rows outside the groups, both encodings, both passes."""
import pytest
import torch

from adapter_ref import check, reference
from test_gpu_dropout import rng_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nf():
    import nf4_base_lora_b200 as nf
    return nf


def make(nf, E, N, K, r, M, dq=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = nf.nf4_quantize(rn(E * N, K) * 0.02, double_quant=dq)
    d = {"A": (rn(E, r, K) / r).bfloat16(), "B": (rn(E, N, r) * 0.05).bfloat16(), "X": rn(M, K).bfloat16(),
         "dY": rn(M, N).bfloat16()}
    return w, nf.nf4_dequantize(w).reshape(E, N, K), d


def offsets_of(counts, first=0):
    off = [first]
    for c in counts:
        off.append(off[-1] + c)
    return off, torch.tensor(off, dtype=torch.int32, device="cuda")


CASES = [
    # E, d_out, d_in, r, rows per expert, first row, rows behind, p, dq
    (1, 128, 64, 8, [1], 0, 0, 0.0, True),
    (2, 128, 128, 8, [1, 1], 0, 0, 0.0, True),
    (4, 136, 192, 4, [3, 0, 1, 2], 2, 3, 0.0, True),              # an expert without rows, rows outside, rank 4
    (8, 264, 320, 16, [16, 15, 17, 1, 0, 9, 8, 7], 0, 5, 0.1, False),
    (3, 8, 64, 1, [5, 0, 70], 1, 1, 0.5, True),                   # the smallest weight
    (5, 512, 256, 64, [127, 128, 129, 0, 1], 0, 0, 0.05, True),   # at the 128-row tile's edges
    (4, 320, 512, 12, [255, 256, 257, 64], 3, 130, 0.25, True),
    (3, 384, 256, 256, [40, 0, 63], 0, 0, 0.5, True),             # largest rank
    (2, 256, 320, 251, [65, 30], 0, 1, 0.0, False),
    (40, 72, 128, 8, [(7 * i) % 23 for i in range(40)], 0, 0, 0.1, True),   # more experts than a warp has lanes
    (70, 64, 64, 8, [1] * 35 + [0] * 34 + [100], 4, 4, 0.0, True),
    (4, 2752, 1024, 16, [700, 1, 300, 530], 0, 9, 0.05, True),    # 256-row tiles
    (6, 1408, 2048, 8, [400, 0, 129, 257, 1000, 6], 5, 0, 0.1, False),
    (8, 4096, 1088, 16, [10, 2, 0, 0, 1, 8, 16, 27], 0, 0, 0.0, True),      # serving, some above 16 rows
    (8, 1096, 4160, 16, [1, 0, 0, 1, 0, 0, 0, 0], 0, 0, 0.0, True),         # one token, two experts
    (130, 72, 128, 8, [(5 * i) % 61 for i in range(130)], 2, 1, 0.1, True),  # more groups than a kernel keeps, 256-token tiles
    (140, 72, 192, 8, [i % 4 for i in range(140)], 0, 3, 0.1, True),         # and 32-token ones
    (300, 64, 64, 8, [0] * 150 + [1200] + [1] * 148 + [700], 0, 0, 0.1, True),  # long groups far apart: summed parts
    (4096, 8, 64, 4, [1 if i % 3 else 0 for i in range(4096)], 0, 7, 0.0, True),  # most experts
    (4096, 8, 64, 4, [0, 1152] * 2048, 0, 0, 0.0, True),                     # the longest list of groups with parts
    (2, 264, 192, 256, [600, 515], 0, 0, 0.25, True),                        # 512-token tiles, largest rank
    (2, 328, 448, 32, [505, 33], 1, 2, 0.0, False),                          # an odd number of blocks
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "E%d_%dx%d_r%d_M%d" % (c[0], c[1], c[2], c[3], sum(c[4])))
def test_grouped_matches_64_bits(nf, case):
    E, N, K, r, counts, first, behind, p, dq = case
    off, offsets = offsets_of(counts, first)
    M = off[-1] + behind
    w, W, d = make(nf, E, N, K, r, M, dq)
    state, s = (31, -7), 8.0 / r
    rng = rng_tensor(state) if p else None
    inside = slice(off[0], off[-1])
    # rows outside the groups hold NaN and must neither be read nor written
    nan = float("nan")
    X, dY = torch.full_like(d["X"], nan), torch.full_like(d["dY"], nan)
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
    for e in range(E):
        if counts[e] == 0:
            assert not dA[e].any() and not dB[e].any()


@pytest.mark.parametrize("counts", [[3, 5, 2], [200, 60, 130], [0, 300, 1]])
def test_one_experts_nan_reaches_only_its_own_rows(nf, counts):
    off, offsets = offsets_of(counts)
    M, r = off[-1], 5
    w, W, d = make(nf, 3, 72, 128, r, M)
    e = max(range(3), key=lambda i: counts[i])
    other = [i for i in range(M) if not off[e] <= i < off[e + 1]]
    clean = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets)
    cg = nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], clean[1], d["dY"], offsets)
    bad = {k: v.clone() for k, v in d.items()}
    bad["A"][e], bad["B"][e] = float("nan"), float("inf")
    bad["X"][off[e]:off[e + 1]], bad["dY"][off[e]:off[e + 1]] = float("inf"), float("nan")
    got = nf.qlora_grouped_fwd(w, bad["A"], bad["B"], 1.0, bad["X"], offsets)
    bg = nf.qlora_grouped_bwd(w, bad["A"], bad["B"], 1.0, bad["X"], got[1], bad["dY"], offsets)
    for a, b in zip((*clean, cg[0]), (*got, bg[0])):
        assert torch.equal(a[other], b[other])
    keep = [i for i in range(3) if i != e]
    assert torch.equal(cg[1][keep], bg[1][keep]) and torch.equal(cg[2][keep], bg[2][keep])


def test_experts_are_the_dense_layer(nf):
    """One expert with all rows is qlora_linear_fwd / _bwd to rounding."""
    M, N, K, r = 200, 256, 320, 16
    w, W, d = make(nf, 1, N, K, r, M)
    off, offsets = offsets_of([M])
    Y, T = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets)
    Y0, T0 = nf.qlora_linear_fwd(w, d["A"][0], d["B"][0], 1.0, d["X"])
    assert (T - T0).abs().max() <= 1e-4 * T0.abs().max()
    assert (Y.double() - Y0.double()).abs().max() <= 2.0 ** -7 * Y0.abs().max()


@pytest.mark.parametrize("counts", [[2, 0, 3], [300, 0, 129]])
def test_accumulation_recomputation_and_single_outputs(nf, counts):
    off, offsets = offsets_of(counts)
    M, r = off[-1], 12
    w, W, d = make(nf, 3, 136, 192, r, M)
    rng = rng_tensor((2, 3))
    _, T = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets, 0.2, rng)
    dX, dA, dB = nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], T, d["dY"], offsets, 0.2, rng)
    _, dA0, dB0 = nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], None, d["dY"], offsets, 0.2, rng, need_dx=False)
    assert torch.equal(dA, dA0) and torch.equal(dB, dB0)
    only = nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, None, None, d["dY"], offsets, 0.2, rng, need_da=False,
                                need_db=False)
    assert torch.equal(only[0], dX)
    a2, b2 = dA.clone(), dB.clone()
    a2[1], b2[1] = 7.0, 7.0                                    # the expert without rows keeps what was there
    nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], T, d["dY"], offsets, 0.2, rng, need_dx=False, dA=a2, dB=b2,
                         accumulate=True)
    assert (a2[1] == 7.0).all() and (b2[1] == 7.0).all()
    for two, one in ((a2, dA), (b2, dB)):
        for e in (0, 2):
            assert ((two[e].double() - 2 * one[e].double()).abs() <= 2.0 ** -8 * 3.1 * one[e].double().abs()
                    + 1e-30).all()


@pytest.mark.parametrize("E,N,K,r,counts,p", [
    (3, 136, 192, 12, [300, 0, 129], 0.2), (3, 2048, 64, 8, [2000, 700, 1300], 0.1), (3, 64, 2048, 256, [600, 0, 300], 0.0),
    (40, 72, 128, 8, [(7 * i) % 23 for i in range(40)], 0.1)])
def test_results_do_not_depend_on_what_else_is_asked_for(nf, E, N, K, r, counts, p):
    """Every choice of gradients, T saved or not, in one workspace that is
    overwritten before each call, in eager calls and in a graph: the same bits."""
    off, offsets = offsets_of(counts)
    M = off[-1]
    w, W, d = make(nf, E, N, K, r, M)
    rng = rng_tensor((8, 9)) if p else None
    ws = torch.empty(nf.qlora_grouped_bwd_workspace_bytes(M, E, N, K, r)
                     + nf.qlora_grouped_fwd_workspace_bytes(M, E, N, K, r), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in (d["dY"], d["X"], d["A"], d["B"])] + [torch.empty(M, r, device="cuda")]

    def call(save=True, **need):
        for t in out:
            t.fill_(7.0)
        ws.fill_(255)
        nf.qlora_grouped_fwd(w, d["A"], d["B"], 0.5, d["X"], offsets, p, rng, Y=out[0], T=out[4], workspace=ws)
        nf.qlora_grouped_bwd(w, d["A"], d["B"], 0.5, d["X"], out[4] if save else None, d["dY"], offsets, p, rng,
                             dX=out[1], dA=out[2], dB=out[3], workspace=ws, **need)
    call()
    first = [t.clone() for t in out]
    for _ in range(4):
        for save in (True, False):
            for dx, da, db in ((1, 1, 1), (0, 1, 1), (1, 0, 1), (1, 1, 0), (0, 0, 1), (0, 1, 0), (1, 0, 0)):
                call(save, need_dx=bool(dx), need_da=bool(da), need_db=bool(db))
                for t, f, asked in zip(out, first, (1, dx, da, db, 1)):
                    assert torch.equal(t, f) if asked else bool((t == 7.0).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call(False)
        call()
    for _ in range(10):
        g.replay()
        assert all(torch.equal(t, f) for t, f in zip(out, first))
    nf.device_status()


def test_a_graph_follows_offsets_that_change(nf):
    E, N, K, r, M = 4, 264, 320, 16, 300
    w, W, d = make(nf, E, N, K, r, M)
    rng = rng_tensor((5, 5))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    Y, T, dX = torch.zeros_like(d["dY"]), torch.zeros((M, r), device="cuda"), torch.zeros_like(d["X"])
    dA, dB = torch.zeros_like(d["A"]), torch.zeros_like(d["B"])
    ws = torch.empty(nf.qlora_grouped_bwd_workspace_bytes(M, E, N, K, r), dtype=torch.uint8, device="cuda")

    def step():
        nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets, 0.1, rng, Y=Y, T=T, workspace=ws)
        nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], T, d["dY"], offsets, 0.1, rng, dX=dX, dA=dA, dB=dB,
                             workspace=ws)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for counts in ([300, 0, 0, 0], [0, 10, 150, 140], [75, 75, 75, 75], [0, 0, 0, 1]):
        off, o = offsets_of(counts)
        offsets.copy_(o)
        g.replay()
        torch.cuda.synchronize()
        ref = reference(W, d["A"], d["B"], d["X"], d["dY"], off, 1.0, 0.1, (5, 5))
        rows = slice(0, off[-1])
        for name, got in (("T", T), ("Y", Y), ("dX", dX)):
            check(got, ref, name, rows)
        check(dA, ref, "dA")
        check(dB, ref, "dB")
    nf.device_status()


def test_calls_on_two_streams_do_not_disturb_each_other(nf):
    E, N, K, r, M = 4, 512, 512, 16, 400
    off, offsets = offsets_of([100, 37, 0, 263])
    sets = [make(nf, E, N, K, r, M, seed=i) for i in range(2)]
    alone = [nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets) for w, _, d in sets]
    grads = [nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], t, d["dY"], offsets)
             for (w, _, d), (_, t) in zip(sets, alone)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = [[], []]
    for _ in range(5):
        for i, (w, _, d) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                y, t = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets)
                res[i].append((y, t, *nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], t, d["dY"], offsets)))
    torch.cuda.synchronize()
    for i in range(2):
        for got in res[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, (*alone[i], *grads[i])))
    nf.device_status()


def test_offsets_that_break_the_rule_are_reported(nf):
    """The kernels clamp every bound into the arrays; the host learns of it."""
    E, N, K, r, M = 3, 128, 128, 8, 64
    w, W, d = make(nf, E, N, K, r, M)
    for off in ([0, 40, 20, 64], [0, 10, 20, 65], [-1, 10, 20, 64], [0, 1 << 30, 20, 64]):
        Y, T = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"],
                                    torch.tensor(off, dtype=torch.int32, device="cuda"))
        with pytest.raises(nf.Nf4Error, match="offsets"):
            nf.device_status()
        nf.device_status()
    off, offsets = offsets_of([20, 20, 24])
    Y, T = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets)
    nf.device_status()
    check(Y, reference(W, d["A"], d["B"], d["X"], d["dY"], off, 1.0), "Y")


def test_an_empty_batch(nf):
    w, W, d = make(nf, 2, 64, 64, 8, 1)
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y, T = nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"][:0], offsets)
    assert Y.shape == (0, 64)
    _, dA, dB = nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"][:0], T, d["dY"][:0], offsets)
    assert not dA.any() and not dB.any()
    # rows, but none in a group
    Y = torch.full((1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    nf.qlora_grouped_fwd(w, d["A"], d["B"], 1.0, d["X"], offsets, Y=Y)
    _, dA, dB = nf.qlora_grouped_bwd(w, d["A"], d["B"], 1.0, d["X"], None, d["dY"], offsets)
    torch.cuda.synchronize()
    assert (Y == 3.0).all() and not dA.any() and not dB.any()


@pytest.mark.parametrize("tokens", [40, 700])
def test_a_mixture_trains_as_its_parts_say(nf, tokens):
    """Routing, two grouped layers with adapter dropout, their backward and the
    optimizer, as a training step runs them: every stage within its bounds of the
    64-bit result for the inputs it had, nothing read back to the host between
    them, and the same step replayed from a graph."""
    E, D, F, r, top, p = 6, 192, 320, 8, 2, 0.1
    M = tokens * top
    g = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    up, down = (nf.nf4_quantize(rn(E * n, k) * 0.05) for n, k in ((F, D), (D, F)))
    Wu, Wd = nf.nf4_dequantize(up).reshape(E, F, D), nf.nf4_dequantize(down).reshape(E, D, F)
    master = [rn(E, r, D) / r, rn(E, F, r) * 0.05, rn(E, r, F) / r, rn(E, D, r) * 0.05]
    start = [m.clone() for m in master]
    param = [m.bfloat16() for m in master]
    moments = [(torch.zeros_like(m), torch.zeros_like(m)) for m in master]
    x, target, router = rn(tokens, D).bfloat16(), rn(tokens, D).bfloat16(), rn(D, E).bfloat16()
    rng = torch.tensor([77, 0], dtype=torch.int64, device="cuda")
    rng2 = torch.tensor([78, 0], dtype=torch.int64, device="cuda")
    s = 1.5
    seen = {}

    def step():
        gate, expert = (x @ router).float().softmax(-1).topk(top)
        flat, order = expert.flatten().sort(stable=True)
        offsets = torch.searchsorted(flat, torch.arange(E + 1, device="cuda"), out_int32=True)
        token = order // top
        xs = x[token].contiguous()
        h, t1 = nf.qlora_grouped_fwd(up, param[0], param[1], s, xs, offsets, p, rng)
        a = torch.nn.functional.silu(h.float()).bfloat16()
        y, t2 = nf.qlora_grouped_fwd(down, param[2], param[3], s, a, offsets, p, rng2)
        scale = gate.flatten()[order].unsqueeze(1)
        out = torch.zeros(tokens, D, device="cuda").index_add_(0, token, y.float() * scale)
        dy = ((out - target.float())[token] * scale).bfloat16()
        da, dA2, dB2 = nf.qlora_grouped_bwd(down, param[2], param[3], s, a, t2, dy, offsets, p, rng2)
        sig = h.float().sigmoid()
        dh = (da.float() * sig * (1 + h.float() * (1 - sig))).bfloat16()
        dx, dA1, dB1 = nf.qlora_grouped_bwd(up, param[0], param[1], s, xs, t1, dh, offsets, p, rng)
        seen.update(off=offsets, xs=xs, h=h, t1=t1, a=a, y=y, t2=t2, dy=dy, da=da, dh=dh, dx=dx,
                    grads=[dA1, dB1, dA2, dB2], before=[q.clone() for q in param])
        nf.lora_adamw_step([(m, q, d, *v) for m, q, d, v in zip(master, param, seen["grads"], moments)], 1e-3)

    def verify():
        torch.cuda.synchronize()
        nf.device_status()
        off = seen["off"].tolist()
        assert off[0] == 0 and off[-1] == M
        b, gr = seen["before"], seen["grads"]
        one = reference(Wu, b[0], b[1], seen["xs"], seen["dh"], off, s, p, (77, 0))
        two = reference(Wd, b[2], b[3], seen["a"], seen["dy"], off, s, p, (78, 0))
        for ref, got in ((one, (seen["t1"], seen["h"], seen["dx"], gr[0], gr[1])),
                         (two, (seen["t2"], seen["y"], seen["da"], gr[2], gr[3]))):
            for name, v in zip(("T", "Y", "dX", "dA", "dB"), got):
                check(v, ref, name)

    def reset():
        for m, m0, q, (m1, m2) in zip(master, start, param, moments):
            m.copy_(m0)
            q.copy_(m0)
            m1.zero_()
            m2.zero_()

    step()
    verify()
    eager = [m.clone() for m in master] + [seen["dx"].clone(), seen["y"].clone()]
    assert all((m != m0).any() for m, m0 in zip(master, start))
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        reset()
        graph.replay()
        verify()
        # the sums of the routed outputs add in any order, all else in one
        assert torch.equal(seen["y"], eager[-1])
    x.copy_(rn(tokens, D))  # other tokens, other offsets
    reset()
    graph.replay()
    verify()
