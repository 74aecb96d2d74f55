"""Pins of the oracle of adapter dropout and expert groups: published answers
of the generator, statistics of the keep decisions, the dense oracle group by
group, and finite differences."""
import math

import numpy as np
import pytest

import oracle
from oracle import adapter


@pytest.mark.parametrize("rounds,counter,key,out", [
    # known answers distributed with the generator's paper
    (7, (0, 0, 0, 0), (0, 0), (0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48)),
    (10, (0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    (10, (0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
])
def test_generator_known_answers(rounds, counter, key, out):
    assert tuple(adapter.philox4x32(counter, key, rounds)) == out


def test_keep_uses_the_generator_as_documented():
    seed, off, p = 0x1234567_89ABCDEF, -5, 0.37
    t = math.floor(p * 32768 + 0.5)
    k = adapter.keep((seed, off), 40, p, first=8 * (1 << 33) + 3)
    for i in range(40):
        elem = 8 * (1 << 33) + 3 + i
        g, o = elem // 8, off % (1 << 64)
        w = adapter.philox4x32((g & 0xFFFFFFFF, g >> 32, o & 0xFFFFFFFF, o >> 32),
                               (seed & 0xFFFFFFFF, seed >> 32), 7)[elem % 8 // 2]
        assert k[i] == (((w >> (16 * (elem % 2))) & 0x7FFF) >= t)


@pytest.mark.parametrize("p", [0.05, 0.5, 0.9])
def test_keep_rate_and_independence(p):
    n = 1 << 20
    q = 1 - adapter.threshold(p) / 32768
    a, b = adapter.keep((7, 0), n, p), adapter.keep((7, 1), n, p)
    sd = math.sqrt(q * (1 - q) / n)
    assert abs(a.mean() - q) < 5 * sd and abs(b.mean() - q) < 5 * sd
    # neighbours within a group, across groups, and across offsets
    for x, y in ((a[:-1], a[1:]), (a[:-8], a[8:]), (a, b)):
        c = np.mean((x - q) * (y - q))
        assert abs(c) < 6 * q * (1 - q) / math.sqrt(len(x))


def test_threshold_rounds_p_to_steps():
    assert adapter.threshold(0.0) == 0 and adapter.threshold(0.5) == 16384
    assert adapter.gain(0.5) == 2.0 and adapter.threshold(2.0 ** -17) == 0


def _case(rng, E, N, K, r, M):
    return (rng.standard_normal((E, N, K)), rng.standard_normal((E, r, K)), rng.standard_normal((E, N, r)),
            rng.standard_normal((M, K)), rng.standard_normal((M, N)))


def test_groups_are_the_dense_layer_row_by_row():
    rng = np.random.default_rng(0)
    W, A, B, X, dY = _case(rng, 4, 6, 8, 3, 11)
    off = [1, 4, 4, 9, 10]
    Y, T = adapter.grouped_forward(W, A, B, X, off, 0.5)
    dX, dA, dB = adapter.grouped_backward(W, A, B, X, dY, off, 0.5)
    for e in range(4):
        g = slice(off[e], off[e + 1])
        y, t = oracle.forward(W[e], A[e], B[e], X[g], 0.5)
        dx, da, db = oracle.backward(W[e], A[e], B[e], X[g], dY[g], 0.5)
        for got, ref in ((Y[g], y), (T[g], t), (dX[g], dx), (dA[e], da), (dB[e], db)):
            np.testing.assert_allclose(got, ref, rtol=1e-12, atol=1e-12)
    assert np.isnan(Y[0]).all() and np.isnan(Y[10]).all() and np.isnan(dX[10]).all()
    assert not dA[1].any() and not dB[1].any()


def test_gradients_match_finite_differences():
    rng = np.random.default_rng(1)
    W, A, B, X, dY = _case(rng, 2, 5, 8, 3, 6)
    off, st, p = [0, 2, 6], (3, 9), 0.4

    def loss(A_, B_, X_):
        return float((adapter.grouped_forward(W, A_, B_, X_, off, 0.7, p, st)[0] * dY).sum())
    dX, dA, dB = adapter.grouped_backward(W, A, B, X, dY, off, 0.7, p, st)
    h = 1e-6
    for which, g in ((0, dA), (1, dB), (2, dX)):
        for i in rng.choice(g.size, 12, replace=False):
            d = [np.zeros_like(A), np.zeros_like(B), np.zeros_like(X)]
            d[which].flat[i] = h
            num = (loss(A + d[0], B + d[1], X + d[2]) - loss(A - d[0], B - d[1], X - d[2])) / (2 * h)
            assert abs(num - g.flat[i]) < 1e-6 * max(1.0, abs(num))


def test_dropped_values_never_matter():
    rng = np.random.default_rng(2)
    W, A, B, X, dY = _case(rng, 1, 5, 16, 3, 4)
    st, p = (11, 0), 0.5
    k = adapter.keep(st, X.size, p).reshape(X.shape)
    X2 = np.where(k, X, np.nan)
    T, T2 = (adapter.grouped_forward(W, A, B, x, [0, 4], 1.0, p, st)[1] for x in (X, X2))
    np.testing.assert_array_equal(T, T2)
