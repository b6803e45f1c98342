"""The router's gradient keeps float32's bits for experts far below the top.

Each dlogit is a product of a score and of factors that are one here up to their own rounding, so its
relative error is the score's.  In units of 2^-24 (half a float32 ulp of a number of mantissa 1), the most
that the steps can add up to:
  softmax, dz = p (0 - dot):  the exponential 5.5 (4 for the hardware's base-2 exponential, whose relative
    error is at most 2^-22, one for the correction of its argument, half for the correction's own error),
    the sum 1 (256 terms below 2^-25 of it), its reciprocal 1, dot 2, two products 2:  11.5
  sigmoid, dz = dw q (1 - q):  the exponential 5.5, its division by 1 + e^-|z| 3 (the hardware's reciprocal,
    one ulp, and a product), 1 - q, the slope and the product with dw 3:  11.5
The bound is 11.5 * 2^-24 = 6.9e-7.  An exponential whose argument x log2(e) is rounded to float32 is off by
up to |x| 2^-24 log2(e) ln 2, 1.3e-6 for the logits from -22.2 to -30 alone.
"""
import numpy as np
import pytest

from _gpu import require_gpu, to_dev, to_host

pytestmark = pytest.mark.gpu

BOUND = 11.5 * 2.0 ** -24


def _far(T, E, seed):
    """Logits from -30 to -22.2, all differences from 0 exact in float32."""
    return np.random.default_rng(seed).uniform(-30.0, -22.2, (T, E)).astype(np.float32)


@pytest.mark.parametrize("E", [16, 64, 100, 256, 500, 1000])
def test_softmax_gradient_far_below_the_top(E):
    torch, fp8bs = require_gpu()
    T = 200
    z = _far(T, E, E)
    z[:, 3] = 0.0
    idx = np.full((T, 1), 3, np.int32)
    dz = to_host(fp8bs.moe_route_backward(to_dev(z), to_dev(idx), to_dev(np.ones((T, 1), np.float32)), normalize=False))
    e = np.exp(z.astype(np.float64))
    p = e / e.sum(1, keepdims=True)
    far = np.delete(np.arange(E), 3)
    rel = np.abs(dz[:, far] / (-p[:, far] * p[:, 3:4]) - 1)
    assert rel.max() <= BOUND, rel.max() * 2 ** 24


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("E,k", [(16, 16), (32, 16), (64, 32), (256, 32), (1000, 32)])
def test_sigmoid_gradient_of_extreme_scores(E, k, sign):
    torch, fp8bs = require_gpu()
    T = 200
    z = sign * np.abs(_far(T, E, E))
    idx = np.stack([np.random.default_rng(t).permutation(E)[:k] for t in range(T)]).astype(np.int32)
    dz = to_host(fp8bs.moe_route_backward(to_dev(z), to_dev(idx), to_dev(np.ones((T, k), np.float32)), fp8bs.SCORE_SIGMOID,
                                          normalize=False))
    t = np.exp(-np.abs(np.take_along_axis(z, idx, 1).astype(np.float64)))
    rel = np.abs(np.take_along_axis(dz, idx, 1) / (t / (1 + t) ** 2) - 1)
    assert rel.max() <= BOUND, rel.max() * 2 ** 24
    rest = np.ones((T, E), bool)
    np.put_along_axis(rest, idx, False, 1)
    assert np.all(dz[rest] == 0)


@pytest.mark.parametrize("score", [0, 1])
def test_largest_finite_logits(score):
    """Float32's extremes are eligible like any other number: scores of 0 and 1, no NaN."""
    torch, fp8bs = require_gpu()
    big = np.finfo(np.float32).max
    z = np.array([[big, -big, 0.0, 1.0], [-big, -big, -big, -big], [100.0, -100.0, 90.0, -90.0], [-big, 3.0, -1e38, 1e38]],
                 np.float32)
    bias = to_dev(np.array([0.0, 3.0, 2.0, 1.0], np.float32)) if score == 1 else None
    for normalize in (True, False):
        idx, w, counts, tokens, loss = fp8bs.moe_route(to_dev(z), 4, score, bias=bias, normalize=normalize, alpha=1.0)
        i, ww = to_host(idx), to_host(w)
        assert np.array_equal(np.sort(i, 1), np.tile(np.arange(4), (4, 1))) and np.all(np.isfinite(ww)) and np.isfinite(float(loss))
        assert np.all(to_host(counts) == 4) and int(tokens) == 4
        dz = to_host(fp8bs.moe_route_backward(to_dev(z), idx, torch.ones_like(w), score, normalize=normalize, alpha=1.0,
                                              counts=counts, tokens=tokens, dloss=torch.ones(1, device="cuda:0")))
        assert np.all(np.isfinite(dz)), dz
