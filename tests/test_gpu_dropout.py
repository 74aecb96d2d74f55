"""Adapter dropout on the GPU: the elementwise operator bit for bit against
the oracle's generator, the layer against 64-bit results."""
import numpy as np
import pytest
import torch

from adapter_ref import check, reference
from oracle import adapter

pytestmark = pytest.mark.gpu

STATES = [(0, 0), (0x1234567_89ABCDEF, 17), (-1, -(1 << 40) - 3)]


@pytest.fixture(scope="module")
def nf():
    import nf4_base_lora_b200 as nf
    return nf


def rng_tensor(state):
    wrap = [((v + (1 << 63)) % (1 << 64)) - (1 << 63) for v in state]
    return torch.tensor(wrap, dtype=torch.int64, device="cuda")


def expected(X, state, p):
    """fp32 product with the fp32 gain, rounded once to the type."""
    k = torch.from_numpy(adapter.keep(state, X.numel(), p).reshape(X.shape))
    x = X.cpu().float() * np.float32(adapter.gain(p))
    return torch.where(k, x, torch.zeros(())).to(X.dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 4096, 100003, (1 << 21) + 5])
def test_elementwise_matches_the_oracle_bit_for_bit(nf, dtype, n):
    for state, p in zip(STATES, (0.05, 0.5, 0.9)):
        X = torch.randn(n, device="cuda").to(dtype)
        out = nf.lora_dropout(X, p, rng_tensor(state))
        assert torch.equal(out.cpu(), expected(X, state, p)), (n, state, p)


def test_elementwise_in_place_shapes_and_no_dropping(nf):
    X = torch.randn(33, 20, device="cuda").bfloat16()
    ref = expected(X, (5, 6), 0.3)
    Y = X.clone()
    assert nf.lora_dropout(Y, 0.3, rng_tensor((5, 6)), out=Y) is Y
    assert torch.equal(Y.cpu(), ref)
    assert torch.equal(nf.lora_dropout(X, 0.0, None), X)
    assert nf.lora_dropout(X[:0], 0.3, rng_tensor((5, 6))).shape == (0, 20)


def test_elementwise_drops_nan_and_infinity(nf):
    X = torch.full((4096,), float("nan"), device="cuda")
    X[::2] = float("inf")
    out = nf.lora_dropout(X, 0.5, rng_tensor((1, 2))).cpu()
    k = torch.from_numpy(adapter.keep((1, 2), 4096, 0.5))
    assert (out[~k] == 0).all() and not torch.isfinite(out[k]).any()


def test_elementwise_beyond_32_bit_offsets(nf):
    n = (1 << 32) + 27
    X = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    nf.lora_dropout(X, 0.5, rng_tensor((3, 4)), out=X)
    for first in (0, (1 << 31) - 40, (1 << 32) - 40, n - 67):
        k = adapter.keep((3, 4), 67, 0.5, first=first)
        assert np.array_equal(X[first:first + 67].float().cpu().numpy(), np.where(k, 2.0, 0.0)), first


def test_the_state_is_read_by_the_kernels(nf):
    """A captured call draws a new mask when the state has changed."""
    X = torch.ones(1 << 16, device="cuda")
    rng = rng_tensor((9, 0))
    out = torch.empty_like(X)
    nf.lora_dropout(X, 0.25, rng, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nf.lora_dropout(X, 0.25, rng, out=out)
        rng[1] += 1
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), expected(X, (9, step), 0.25)), step


# ------------------------------------------------------------------ the layer
def make(nf, N, K, M, r, dq=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = nf.nf4_quantize(rn(N, K) * 0.02, double_quant=dq)
    d = {"A": (rn(r, K) / r).bfloat16(), "B": (rn(N, r) * 0.05).bfloat16(), "X": rn(M, K).bfloat16(),
         "dY": rn(M, N).bfloat16()}
    return w, nf.nf4_dequantize(w), d


CASES = [
    # d_out, d_in, M, r, p, dq
    (128, 64, 1, 8, 0.1, True),
    (136, 192, 3, 4, 0.5, True),           # rank off the multiple of 8
    (512, 512, 16, 8, 0.1, True),
    (8, 64, 17, 1, 0.3, True),             # smallest weight, rank 1
    (264, 320, 130, 12, 0.05, False),
    (512, 768, 300, 128, 0.25, True),
    (384, 1024, 200, 192, 0.1, True),
    (384, 256, 40, 256, 0.5, True),        # largest rank
    (256, 256, 33, 251, 0.5, False),
    (4736, 4800, 2000, 16, 0.05, True),    # 256-row tiles, ragged rows and columns
    (4096, 4096, 1100, 64, 0.1, True),
]


@pytest.mark.parametrize("N,K,M,r,p,dq", CASES)
def test_layer_matches_64_bits(nf, N, K, M, r, p, dq):
    w, W, d = make(nf, N, K, M, r, dq)
    state, s = (77, 1 << 35), 16.0 / r
    rng = rng_tensor(state)
    Y, T = nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], s, d["X"], p, rng)
    dX, dA, dB = nf.qlora_linear_dropout_bwd(w, d["A"], d["B"], s, d["X"], T, d["dY"], p, rng)
    torch.cuda.synchronize()
    nf.device_status()
    ref = reference(W[None], d["A"][None], d["B"][None], d["X"], d["dY"], [0, M], s, p, state)
    for name, got in (("T", T), ("Y", Y), ("dX", dX), ("dA", dA[None]), ("dB", dB[None])):
        check(got, ref, name)


@pytest.mark.parametrize("M", [5, 200])
def test_layer_uses_the_elementwise_mask_and_p_zero_is_the_plain_layer(nf, M):
    w, W, d = make(nf, 256, 320, M, 16)
    rng = rng_tensor((4, 2))
    _, T = nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], 1.0, d["X"], 0.5, rng)
    D = nf.lora_dropout(d["X"], 0.5, rng)  # exact: the gain is 2
    Tm = D.double() @ d["A"].double().T
    assert (T.double() - Tm).abs().max() <= 320 * 2.0 ** -23 * float((D.double().abs() @ d["A"].double().abs().T).max())
    ref = reference(W[None], d["A"][None], d["B"][None], d["X"], d["dY"], [0, M], 1.0)
    Y, T = nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], 1.0, d["X"], 0.0, None)
    dX, dA, dB = nf.qlora_linear_dropout_bwd(w, d["A"], d["B"], 1.0, d["X"], T, d["dY"], 0.0, None)
    for name, got in (("T", T), ("Y", Y), ("dX", dX), ("dA", dA[None]), ("dB", dB[None])):
        check(got, ref, name)


@pytest.mark.parametrize("M", [9, 150])
def test_dropped_nan_stays_out_of_the_adapter(nf, M):
    w, W, d = make(nf, 128, 256, M, 8)
    state, p = (21, 5), 0.5
    k = torch.from_numpy(adapter.keep(state, M * 256, p).reshape(M, 256)).cuda()
    bad = torch.where(k, d["X"], torch.full_like(d["X"], float("nan")))
    rng = rng_tensor(state)
    _, T = nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], 2.0, d["X"], p, rng)
    _, Tb = nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], 2.0, bad, p, rng)
    assert torch.equal(T, Tb)
    a = nf.qlora_linear_dropout_bwd(w, d["A"], d["B"], 2.0, d["X"], T, d["dY"], p, rng)
    b = nf.qlora_linear_dropout_bwd(w, d["A"], d["B"], 2.0, bad, T, d["dY"], p, rng)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # an infinite adapter reaches dX at kept elements only
    A = d["A"].clone()
    A[3, 100] = float("inf")
    dX = nf.qlora_linear_dropout_bwd(w, A, d["B"], 2.0, d["X"], T, d["dY"], p, rng, need_da=False, need_db=False)[0]
    assert torch.equal(torch.isfinite(dX[:, 100]), ~k[:, 100])
    assert torch.isfinite(dX[:, :100]).all() and torch.isfinite(dX[:, 101:]).all()


@pytest.mark.parametrize("M,r", [(7, 5), (200, 12), (1500, 16)])
def test_accumulation_recomputation_and_single_outputs(nf, M, r):
    w, W, d = make(nf, 256, 320, M, r)
    rng, s = rng_tensor((8, 8)), 0.5
    _, T = nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], s, d["X"], 0.2, rng)
    args = (w, d["A"], d["B"], s, d["X"])
    dX, dA, dB = nf.qlora_linear_dropout_bwd(*args, T, d["dY"], 0.2, rng)
    _, dA0, dB0 = nf.qlora_linear_dropout_bwd(*args, None, d["dY"], 0.2, rng, need_dx=False)
    assert torch.equal(dA, dA0) and torch.equal(dB, dB0)       # T recomputed is T
    only = nf.qlora_linear_dropout_bwd(w, d["A"], d["B"], s, None, None, d["dY"], 0.2, rng, need_da=False,
                                       need_db=False)
    assert torch.equal(only[0], dX) and only[1] is None and only[2] is None
    a2, b2 = dA.clone(), dB.clone()
    nf.qlora_linear_dropout_bwd(*args, T, d["dY"], 0.2, rng, need_dx=False, dA=a2, dB=b2, accumulate=True)
    # the sum of the old value and an unrounded gradient that rounds to it: 2 dA off by its own rounding and one more
    for two, one in ((a2, dA), (b2, dB)):
        assert ((two.double() - 2 * one.double()).abs() <= 2.0 ** -8 * 3.1 * one.double().abs() + 1e-30).all()


def test_repeated_calls_agree_and_a_graph_replays_the_step(nf):
    M, r, p = 300, 16, 0.1
    w, W, d = make(nf, 512, 640, M, r)
    rng = rng_tensor((6, 0))
    ws = torch.empty(nf.qlora_linear_dropout_bwd_workspace_bytes(M, 512, 640, r), dtype=torch.uint8, device="cuda")
    out = {k: torch.empty_like(d[v]) for k, v in (("dX", "X"), ("dA", "A"), ("dB", "B"), ("Y", "dY"))}
    T = torch.empty((M, r), device="cuda")

    def step():
        nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], 1.0, d["X"], p, rng, Y=out["Y"], T=T, workspace=ws)
        nf.qlora_linear_dropout_bwd(w, d["A"], d["B"], 1.0, d["X"], T, d["dY"], p, rng, dX=out["dX"], dA=out["dA"],
                                    dB=out["dB"], workspace=ws)
    runs = []
    for i in range(3):
        rng[1] = i
        step()
        runs.append([t.clone() for t in (*out.values(), T)])
    assert not torch.equal(runs[0][-1], runs[1][-1])
    rng[1] = 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
        rng[1] += 1
    for i in range(3):
        for t in out.values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*out.values(), T), runs[i])), i
    nf.device_status()


def test_an_empty_batch(nf):
    w, W, d = make(nf, 64, 64, 1, 8)
    rng = rng_tensor((1, 1))
    Y, T = nf.qlora_linear_dropout_fwd(w, d["A"], d["B"], 1.0, d["X"][:0], 0.1, rng)
    assert Y.shape == (0, 64) and T.shape == (0, 8)
    _, dA, dB = nf.qlora_linear_dropout_bwd(w, d["A"], d["B"], 1.0, d["X"][:0], T, d["dY"][:0], 0.1, rng)
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("M,r", [(300, 16), (19200, 16), (19200, 136)])
def test_the_adapters_sum_keeps_32_bits(nf, M, r):
    """T of a wide layer, few and many tiles, one set of accumulators and several.
    A tensor-core addition truncates: at most one unit (2^-23) of the running sum,
    half of one on average, and an accumulator takes at most 1024 products, 16 an
    addition, so that T is off by about 64 2^-24 of its norm at most (688 additions
    in a row would be 688 2^-24)."""
    N, K = 64, 11008
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = nf.nf4_quantize(rn(N, K) * 0.02)
    A, B, X = (rn(r, K) / r).bfloat16(), (rn(N, r) * 0.05).bfloat16(), rn(M, K).bfloat16()
    _, T = nf.qlora_linear_dropout_fwd(w, A, B, 2.0, X, 0.0, None)
    rows = torch.arange(0, M, max(1, M // 256), device="cuda")
    ref = 2.0 * X[rows].double() @ A.double().T
    err = (T[rows].double() - ref).norm() / ref.norm()
    assert err <= 64 * 2.0 ** -24, float(err)
