"""Terms of the router's gradient that cancel do so without leaving their rounding behind.

Normalised weights do not change when all chosen scores grow together, so a part that all of a token's dw
share has no effect (with one choice, all of dw), and under softmax scores experts that were not chosen get
nothing from the weights.  The probabilities of the loss sum to one, so a part that all experts' loads share
has no effect.  (Up to the 1e-20 that is added to the sums.)  What is left has to be as exact as if the
shared part were not there: differences below 4 x 2^-24 of the larger result, two roundings on either side.
"""
import numpy as np
import pytest

from oracle import route
from _gpu import require_gpu, to_dev, to_host
from test_route_gpu import _logits

pytestmark = pytest.mark.gpu

SIZES = [(16, 1), (30, 3), (64, 6), (100, 8), (256, 8), (300, 8), (600, 20), (1000, 32)]


def _same(a, b):
    return np.all(np.abs(a - b) <= 4 * 2.0 ** -24 * np.maximum(np.abs(a), np.abs(b)) + 1e-25)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,k", SIZES)
def test_a_shared_part_of_dw_has_no_effect(E, k, score):
    torch, fp8bs = require_gpu()
    T = 150
    z = to_dev(_logits(T, E, E))
    kw = dict(score=score, scale=2.5, alpha=1e-3)
    idx, w, counts, tokens, loss = fp8bs.moe_route(z, k, **kw)
    loss_kw = dict(counts=counts, tokens=tokens, dloss=torch.ones(1, device="cuda:0"))
    dw = np.random.default_rng(E).integers(-64, 64, (T, k)).astype(np.float32) / 64       # dw + 1024 is exact
    for extra in ({}, loss_kw):
        plain, shifted = (to_host(fp8bs.moe_route_backward(z, idx, to_dev(d), **kw, **extra)) for d in (dw, dw + 1024))
        assert _same(plain, shifted), np.abs(plain - shifted).max()
    if k == 1:
        alone = to_host(fp8bs.moe_route_backward(z, idx, to_dev(0 * dw), **kw, **loss_kw))
        assert _same(plain, alone), np.abs(plain - alone).max()


@pytest.mark.parametrize("E,k", SIZES)
def test_softmax_weights_give_nothing_to_experts_not_chosen(E, k):
    torch, fp8bs = require_gpu()
    T = 150
    z = to_dev(_logits(T, E, E))
    idx, w = fp8bs.moe_route(z, k)
    dw = np.random.default_rng(E).standard_normal((T, k)).astype(np.float32)
    dz = to_host(fp8bs.moe_route_backward(z, idx, to_dev(dw)))
    chosen = np.zeros((T, E), bool)
    np.put_along_axis(chosen, to_host(idx).astype(np.int64), True, 1)
    assert np.all(np.abs(dz[~chosen]) <= 1e-18)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,k", SIZES)
def test_a_shared_part_of_the_loads_has_no_effect(E, k, score):
    """Loads of 5000 and a few more or less: the gradient of the few, to 2e-6 of its largest, as the float64 form
    has it (seven roundings of the sums and products, 2^-24 each, four times over)."""
    torch, fp8bs = require_gpu()
    T = 150
    z = _logits(T, E, E)
    counts = 5000 + np.random.default_rng(E).integers(-5, 6, (1, E))
    tokens = np.array([5000 * E // k])
    none = np.full((T, k), -1, np.int32)
    got = to_host(fp8bs.moe_route_backward(to_dev(z), to_dev(none), torch.zeros((T, k), device="cuda:0"), score, alpha=0.5,
                                           counts=to_dev(counts.astype(np.int32)), tokens=to_dev(tokens.astype(np.int32)),
                                           dloss=torch.ones(1, device="cuda:0")))
    g = 0.5 * E * counts[0] / k / tokens[0] ** 2
    ref = np.zeros((T, E))
    for t in range(T):
        s, _ = route.scores(z[t].astype(np.float64), score)
        p = s / s.sum()
        dp = g - (p * g).sum()
        ref[t] = p * dp if score == 0 else s * (1 - s) * dp / s.sum()
    big = np.abs(ref).max(axis=1, keepdims=True)
    assert np.all(np.abs(got - ref) <= 2e-6 * big), (np.abs(got - ref) / big).max()
    even = to_host(fp8bs.moe_route_backward(to_dev(z), to_dev(none), torch.zeros((T, k), device="cuda:0"), score, alpha=0.5,
                                            counts=torch.full((1, E), 5000, dtype=torch.int32, device="cuda:0"),
                                            tokens=to_dev(tokens.astype(np.int32)), dloss=torch.ones(1, device="cuda:0")))
    assert np.all(np.abs(even) <= 1e-18)
