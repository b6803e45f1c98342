"""The training operators' oracle against central differences in float64.

Each gradient is checked as the derivative of <output, weights> along random directions: the difference
quotient's error is the rounding of float64 sums divided by the step, and the step's square times a third
derivative; both stay under 1e-6 of the scale at a step of 1e-5 and values near one."""
import numpy as np
import pytest

from oracle import train

STEP, TOL = 1e-5, 1e-6


def _slope(f, x, direction):
    return (f(x + STEP * direction) - f(x - STEP * direction)) / (2 * STEP)


@pytest.mark.parametrize("seed", range(3))
def test_rmsnorm_gradient(seed):
    rng = np.random.default_rng(seed)
    M, K, eps = 3, 16, 1e-3
    r, gain, dy, dres = rng.standard_normal((M, K)), rng.standard_normal(K), rng.standard_normal((M, K)), rng.standard_normal((M, K))
    _, rstd = train.rmsnorm(r, gain, eps)
    dx, mag, dgain, _ = train.rmsnorm_backward(dy, r, gain, rstd, dres)

    def value(x):
        return float((train.rmsnorm(x, gain, eps)[0] * dy).sum() + (x * dres).sum())

    v = rng.standard_normal((M, K))
    assert abs(_slope(value, r, v) - float((dx * v).sum())) < TOL * mag.sum()
    u = rng.standard_normal(K)
    slope = _slope(lambda g: float((train.rmsnorm(r, g, eps)[0] * dy).sum()), gain, u)
    assert abs(slope - float((dgain * u).sum())) < TOL * np.abs(dy).sum()


def test_swiglu_gradient():
    rng = np.random.default_rng(0)
    M, I = 4, 8
    h, dv, v = 2 * rng.standard_normal((M, 2 * I)), rng.standard_normal((M, I)), rng.standard_normal((M, 2 * I))

    def value(x):
        g, u = x[:, :I], x[:, I:]
        return float((g / (1 + np.exp(-g)) * u * dv).sum())

    dh, mag = train.swiglu_backward(h, dv, I)
    assert abs(_slope(value, h, v) - float((dh * v).sum())) < TOL * mag.sum()


def test_swiglu_gradient_far_from_zero():
    """sigma(g) (1 + g sigma(-g)) is 1 far above zero and (1 + g) e^g far below."""
    g = np.array([[-300.0, -100.0, 100.0, 300.0]])
    dh, _ = train.swiglu_backward(np.concatenate([g, np.ones((1, 4))], axis=1), np.ones((1, 4)), 4)
    assert np.allclose(dh[0, :4], [-299 * np.exp(-300.0), -99 * np.exp(-100.0), 1.0, 1.0], rtol=1e-12)
    assert np.allclose(dh[0, 4:], [-300 * np.exp(-300.0), -100 * np.exp(-100.0), 100.0, 300.0], rtol=1e-12)


def test_sorting_gradients():
    rng = np.random.default_rng(1)
    T, k, N, rows = 5, 3, 6, 20
    row_of = rng.permutation(rows)[:T * k].reshape(T, k)
    row_of[2, 1] = -1
    x, y, w, dout = rng.standard_normal((T, N)), rng.standard_normal((rows, N)), rng.standard_normal((T, k)), rng.standard_normal((T, N))
    d = rng.standard_normal((rows, N))

    def combined(yy, ww):
        out = np.zeros((T, N))
        for t in range(T):
            for j in range(k):
                if row_of[t, j] >= 0:
                    out[t] += ww[t, j] * yy[row_of[t, j]]
        return float((out * dout).sum())

    def dispatched(xx):
        out = np.zeros((rows, N))
        for t in range(T):
            for j in range(k):
                if row_of[t, j] >= 0:
                    out[row_of[t, j]] = xx[t]
        return float((out * d).sum())

    dy, dw, mag = train.combine_backward(dout, y, row_of, w, rows)
    v, u, z = rng.standard_normal(y.shape), rng.standard_normal(w.shape), rng.standard_normal(x.shape)
    assert abs(_slope(lambda q: combined(q, w), y, v) - float((dy * v).sum())) < TOL * mag.sum()
    assert abs(_slope(lambda q: combined(y, q), w, u) - float((dw * u).sum())) < TOL * mag.sum()
    dx, m = train.dispatch_backward(d, row_of)
    assert abs(_slope(dispatched, x, z) - float((dx * z).sum())) < TOL * m.sum()
    assert np.all(dy[np.setdiff1d(np.arange(rows), row_of)] == 0) and dw[2, 1] == 0


def test_weight_gradient():
    rng = np.random.default_rng(2)
    N, K, R, offsets = 4, 3, 12, [0, 5, 5, 10]
    a, b = rng.standard_normal((N, R)), rng.standard_normal((K, R))
    d, _ = train.grouped_wgrad(a, b, offsets)
    w, v = rng.standard_normal((3, N, K)), rng.standard_normal((3, N, K))

    def value(x):      # the outputs' gradients a are those of <x b, a> over each expert's columns
        return float(sum((a[:, offsets[g]:offsets[g + 1]] * (x[g] @ b[:, offsets[g]:offsets[g + 1]])).sum() for g in range(3)))

    assert abs(_slope(value, w, v) - float((d * v).sum())) < TOL * np.abs(a).sum() * 3
    assert np.all(d[1] == 0)
