"""CPU oracle of the adapter's dropout and of the layer of a mixture of experts.

TEST INFRASTRUCTURE ONLY, as the rest of this package: plain numpy in 64 bits,
no code shared with the CUDA path.

Dropout of the adapter's input, D = keep .* X * gain with gain = 2^15 / (2^15 - t),
t = floor(p 2^15 + 1/2):

  forward   T = s D A^T,  Y = X W_hat^T + T B^T
  backward  V = s dY B,  dX = dY W_hat + gain keep .* (V A),  dA = V^T D,  dB = dY^T T

Generator: Philox4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
as easy as 1, 2, 3", SC 2011) with 7 rounds.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence, Tuple

import numpy as np

from . import _f64

MASK32 = (1 << 32) - 1


def philox4x32(counter: Sequence[int], key: Sequence[int], rounds: int) -> List[int]:
    """One block of the generator on Python integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & MASK32, (a >> 32) ^ c[3] ^ k[1], a & MASK32]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    return c


def threshold(p: float) -> int:
    return math.floor(p * 32768 + 0.5)


def gain(p: float) -> float:
    return 32768.0 / (32768 - threshold(p))


def keep(state: Tuple[int, int], n: int, p: float, first: int = 0) -> np.ndarray:
    """Keep decisions (bool) of the flat elements first .. first + n - 1 for
    state = (seed, offset), both taken modulo 2^64."""
    t = threshold(p)
    g0 = first // 8
    groups = np.arange(g0, (first + n + 7) // 8, dtype=np.uint64)
    u = np.uint64
    seed, off = (int(v) % (1 << 64) for v in state)
    c = [groups & u(MASK32), groups >> u(32), np.full_like(groups, off & MASK32), np.full_like(groups, off >> 32)]
    k = [seed & MASK32, seed >> 32]
    for _ in range(7):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> u(32)) ^ c[1] ^ u(k[0]), b & u(MASK32), (a >> u(32)) ^ c[3] ^ u(k[1]), a & u(MASK32)]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    halves = []
    for w in c:
        halves += [w & u(0x7FFF), (w >> u(16)) & u(0x7FFF)]
    bits = np.stack(halves, axis=1).reshape(-1)[first - 8 * g0:][:n]
    return bits >= t


def dropout(X, state, p: float) -> np.ndarray:
    X = _f64(X)
    return np.where(keep(state, X.size, p).reshape(X.shape), X * gain(p), 0.0)


def _dropped(M: np.ndarray, mask: Optional[np.ndarray], p: float) -> np.ndarray:
    return M if mask is None else np.where(mask, M * gain(p), 0.0)


def _mask(shape, state, p: float) -> Optional[np.ndarray]:
    return keep(state, int(np.prod(shape)), p).reshape(shape) if threshold(p) else None


def grouped_forward(W_hat, A, B, X, offsets, scaling: float, p: float = 0.0, state=(0, 0)):
    """(Y, T) with W_hat [E, d_out, d_in], A [E, r, d_in], B [E, d_out, r];
    rows outside the groups are NaN (they have no value)."""
    W_hat, A, B, X = map(_f64, (W_hat, A, B, X))
    D = _dropped(X, _mask(X.shape, state, p), p)
    Y = np.full((X.shape[0], W_hat.shape[1]), np.nan)
    T = np.full((X.shape[0], A.shape[1]), np.nan)
    for e in range(W_hat.shape[0]):
        g = slice(offsets[e], offsets[e + 1])
        T[g] = scaling * (D[g] @ A[e].T)
        Y[g] = X[g] @ W_hat[e].T + T[g] @ B[e].T
    return Y, T


def grouped_backward(W_hat, A, B, X, dY, offsets, scaling: float, p: float = 0.0, state=(0, 0)):
    """(dX, dA, dB) of <dY, Y> for the forward above."""
    W_hat, A, B, X, dY = map(_f64, (W_hat, A, B, X, dY))
    mask = _mask(X.shape, state, p)
    D = _dropped(X, mask, p)
    dX = np.full(X.shape, np.nan)
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for e in range(W_hat.shape[0]):
        g = slice(offsets[e], offsets[e + 1])
        T, V = scaling * (D[g] @ A[e].T), scaling * (dY[g] @ B[e])
        dX[g] = dY[g] @ W_hat[e] + _dropped(V @ A[e], None if mask is None else mask[g], p)
        dA[e], dB[e] = V.T @ D[g], dY[g].T @ T
    return dX, dA, dB
