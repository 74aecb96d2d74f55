"""64-bit results of the dropout and grouped layers with element-wise error
bounds, for the GPU tests.

The bounds count the roundings of the kernels' arithmetic.  A product of two
bfloat16 values is exact in fp32; a sum of n of them is off by at most
n 2^-23 S, S the sum of the magnitudes (one rounding or truncation per
addition).  With |.| element-wise:

  T = s gain sum      bT  = (K 2^-23 + 2^-22) s gain |D||A|^T   (the factor's and the product's roundings)
  pair of T           2^-16 |T|   (two bfloat16 halves: 2^-8 of 2^-8)
  Y                   2^-8 |Y| + (K + 2 r) 2^-23 (|X||W|^T + |T||B|^T) + (bT + 2^-16 |T|) |B|^T

and alike for V, dX, dA (sum over a group's rows, halves added separately) and
dB.  The last rounding is of a value that is off by the rest, so the whole
bound is multiplied by 1 + 2^-7."""
import numpy as np
import torch

from oracle import adapter

OUT = 2.0 ** -8
ACC = 2.0 ** -23
PAIR = 2.0 ** -16


def keep_mask(shape, state, p):
    n = int(np.prod(shape))
    return torch.from_numpy(adapter.keep(state, n, p).reshape(shape)).cuda()


def reference(W, A, B, X, dY, offsets, s, p=0.0, state=(0, 0)):
    """{name: (value, bound)}; W [E, N, K] and the adapters [E, ...] in any
    type; rows outside the groups are NaN in value and bound."""
    W, A, B, X, dY = (t.double() for t in (W, A, B, X, dY))
    E, N, K = W.shape
    r = A.shape[1]
    t = adapter.threshold(p)
    g = adapter.gain(p)
    s = float(np.float32(s))
    k = keep_mask(X.shape, state, p) if t else torch.ones_like(X, dtype=torch.bool)
    nan = float("nan")
    out = {"Y": torch.full_like(dY, nan), "T": torch.full((X.shape[0], r), nan, dtype=torch.float64, device=X.device),
           "dX": torch.full_like(X, nan), "dA": torch.zeros_like(A), "dB": torch.zeros_like(B)}
    tol = {n: v.clone() for n, v in out.items()}
    for e in range(E):
        i, j = offsets[e], offsets[e + 1]
        if i == j:
            continue
        w, a, b, x, dy, kk = W[e], A[e], B[e], X[i:j], dY[i:j], k[i:j]
        d = torch.where(kk, x * g, 0.0)
        T, V = s * (d @ a.T), s * (dy @ b)
        aT, aV = abs(s) * (d.abs() @ a.abs().T), abs(s) * (dy.abs() @ b.abs())
        bT, bV = (K * ACC + 2 * 2.0 ** -23) * aT, (N * ACC + 2 * 2.0 ** -23) * aV
        eT, eV = bT + PAIR * T.abs(), bV + PAIR * V.abs()
        va, m = V @ a, j - i
        res = {"T": (T, bT), "Y": (x @ w.T + T @ b.T,
                                   (K + 2 * r) * ACC * (x.abs() @ w.abs().T + T.abs() @ b.abs().T) + eT @ b.abs().T),
               "dX": (dy @ w + torch.where(kk, g * va, 0.0),
                      (N + 2 * r) * ACC * (dy.abs() @ w.abs() + g * (V.abs() @ a.abs())) + g * (eV @ a.abs())),
               "dA": (V.T @ d, 2 * (m + 64) * ACC * (V.abs().T @ d.abs()) + eV.T @ d.abs()),
               "dB": (dy.T @ T, 2 * (m + 64) * ACC * (dy.abs().T @ T.abs()) + dy.abs().T @ eT)}
        for n, (v, bound) in res.items():
            at = e if n in ("dA", "dB") else slice(i, j)
            out[n][at] = v
            tol[n][at] = bound if n == "T" else (bound + OUT * v.abs()) * (1 + 2.0 ** -7)
    return {n: (out[n], tol[n]) for n in out}


def check(got, ref, name, rows=None):
    """Every element within its bound (rows: a slice of rows that have values)."""
    v, tol = ref[name]
    if rows is not None:
        got, v, tol = got[rows], v[rows], tol[rows]
    if v.numel() == 0:
        return
    err = (got.double() - v).abs()
    bad = ~(err <= tol + 1e-30)
    assert not bad.any(), "%s: %d of %d elements off, worst %.3g against a bound of %.3g at %s" % (
        name, int(bad.sum()), bad.numel(), float(torch.nan_to_num(err - tol, nan=1e30).max()),
        float(tol.reshape(-1)[torch.argmax(torch.nan_to_num(err - tol, nan=1e30))]), bad.nonzero()[0].tolist())
    # and, much closer than the worst case, on average
    scale = float(v.abs().mean())
    mean = float(err.mean())
    assert mean <= 2.5e-3 * scale + 1e-30, "%s: mean error %.3g of a mean magnitude %.3g" % (name, mean, scale)
