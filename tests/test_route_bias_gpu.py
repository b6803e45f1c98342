"""The router with a selection bias, as a model with auxiliary-loss-free balancing trains and serves it:
statistics and gradient, masked and ineligible experts, BF16 logits, many experts and choices, ties; and
the gradient's instances that other tests do not reach.  Tolerances as in test_route_gpu.py; where a token
has one eligible expert its gradient cancels to zero, so the gradient's bound, 2e-5 of the sum of the terms'
magnitudes, is taken from the terms themselves."""
import numpy as np
import pytest

from oracle import route
from _gpu import require_gpu, to_dev, to_host
from test_route_gpu import SEQS, _dev, _logits

pytestmark = pytest.mark.gpu


def _inputs(T, E, k, bf16, holes, seed):
    """Logits, bias and mask such that float32 rounding cannot move the choice: among a token's k + 1 largest
    biased keys, those that are not the same logit with the same bias are 1e-6 apart."""
    rng = np.random.default_rng(seed)
    z = _logits(8 * T + 8, E, seed, bf16)
    bias = (np.round(rng.standard_normal(E) * 100) * 1e-3).astype(np.float32)
    if holes:
        z[rng.random(z.shape) < 0.05] = -np.inf
        z[rng.random(z.shape) < 0.02] = np.nan
        z[5::17, 2:] = np.nan
        z[7::19] = -np.inf
    with np.errstate(over="ignore"):
        key = np.where(np.isnan(z) | np.isneginf(z), -np.inf, 1 / (1 + np.exp(-z.astype(np.float64))) + bias)
    top = -np.sort(-key, axis=1)[:, :k + 1]
    with np.errstate(invalid="ignore"):
        gap = top[:, :-1] - top[:, 1:]
    z = z[np.all(~(gap <= 1e-6) | (gap == 0), axis=1)][:T]
    assert len(z) == T
    valid = (rng.random(T) > 0.1).astype(np.uint8) if holes else np.ones(T, np.uint8)
    return z, bias, valid


def _gradient_bound(z, idx, dw, counts, tokens, dloss, valid, seq, normalize, scale, alpha):
    """2e-5 of sum |terms| of each d logit: sigmoid, dz = s (1 - s) (d weights + d loss)."""
    T, E = z.shape
    k = idx.shape[1]
    seq = [0, T] if seq is None else seq
    bound = np.zeros((T, E))
    for q in range(len(seq) - 1):
        g = dloss * alpha / (len(seq) - 1) * E * counts[q] / k / max(tokens[q], 1) ** 2
        for t in range(seq[q], seq[q + 1]):
            if not valid[t]:
                continue
            s, _ = route.scores(z[t].astype(np.float64), 1)
            total = s.sum() + 1e-20
            m = (g + (s * g).sum() / total) / total
            sel = idx[t] >= 0
            i, d = idx[t][sel], np.abs(dw[t][sel])
            chosen = s[i].sum() + 1e-20
            m[i] += scale * ((d + (d * s[i]).sum() / chosen) / chosen if normalize else d)
            bound[t] = 2e-5 * s * (1 - s) * m
    return bound


@pytest.mark.parametrize("holes", [False, True])
@pytest.mark.parametrize("T,E,k,bf16", [(33, 13, 4, False), (60, 64, 6, True), (50, 64, 20, False), (120, 256, 8, False),
                                        (90, 256, 8, True), (40, 200, 17, True), (60, 300, 8, False), (40, 600, 12, True),
                                        (30, 1024, 32, False)])
@pytest.mark.parametrize("seqs", ["one", "odd"])
def test_bias_with_statistics_and_gradient(T, E, k, bf16, holes, seqs):
    torch, fp8bs = require_gpu()
    z, bias, valid = _inputs(T, E, k, bf16, holes, T + E)
    seq = SEQS[seqs](T)
    dseq = None if seq is None else to_dev(np.array(seq, np.int32))
    zd, vd, bd = _dev(torch, z, bf16), to_dev(valid), to_dev(bias)
    kw = dict(score=1, scale=2.5)
    ri, rw, rc, rt, rl = route.route(z, k, bias=bias.astype(np.float64), valid=valid, seq=seq, alpha=0.7, **kw)
    idx, w = fp8bs.moe_route(zd, k, bias=bd, valid=vd, **kw)
    assert np.array_equal(to_host(idx), ri) and np.allclose(to_host(w), rw, rtol=1e-5, atol=1e-30)
    idx, w, counts, tokens, loss = fp8bs.moe_route(zd, k, bias=bd, valid=vd, seq=dseq, alpha=0.7, **kw)
    assert np.array_equal(to_host(idx), ri) and np.allclose(to_host(w), rw, rtol=1e-5, atol=1e-30)
    assert np.array_equal(to_host(counts), rc) and np.array_equal(to_host(tokens), rt)
    assert np.allclose(to_host(loss), rl, rtol=2e-5)
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    dw[ri < 0] = np.nan
    for normalize in (True, False):
        got = to_host(fp8bs.moe_route_backward(zd, idx, to_dev(dw), valid=vd, seq=dseq, counts=counts, tokens=tokens, alpha=0.7,
                                               dloss=to_dev(np.array([1.3], np.float32)), normalize=normalize, **kw))
        ref = route.backward(z, ri, np.nan_to_num(dw), 1.3, valid=valid, seq=seq, alpha=0.7, normalize=normalize, **kw)
        tol = _gradient_bound(z, ri, dw, rc, rt, 1.3, valid, seq, normalize, 2.5, 0.7)
        tol += (2.0 ** -8 * (np.abs(ref) + tol) if bf16 else 0) + 1e-30
        assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()
        assert np.all(got[valid == 0] == 0) and np.all(got[~np.isfinite(z)] == 0)


@pytest.mark.parametrize("stats", [False, True])
@pytest.mark.parametrize("E,k", [(16, 4), (40, 4), (40, 16), (64, 20), (100, 8), (256, 8), (300, 8), (1000, 32)])
def test_ties_and_close_keys_beyond_the_candidates(E, k, stats):
    """Equal logits: with equal biases every key ties (lower indices win); with biases that rise by a
    float32 ulp all of up to 168 keys lie within the margin of the candidates' bound, more than their list
    holds, and the largest win.  Every other token is an ordinary one."""
    torch, fp8bs = require_gpu()
    T = 10
    order = np.random.default_rng(E).permutation(E)
    for bias in (np.full(E, 0.25, np.float32), (np.argsort(order) * 2.0 ** -24).astype(np.float32)):
        z = np.zeros((T, E), np.float32)                 # sigmoid(0) = 0.5, and 0.5 + i 2^-24 is exact
        z[1::2, : k + 2] = 1.0 + np.arange(k + 2) * 0.125
        key = np.where(z == 0, 0.5, 1 / (1 + np.exp(-z.astype(np.float64)))) + bias
        ref = np.argsort(-key, axis=1, kind="stable")[:, :k]
        got = fp8bs.moe_route(to_dev(z), k, fp8bs.SCORE_SIGMOID, bias=to_dev(bias), alpha=0.1 if stats else None)
        assert np.array_equal(to_host(got[0]), ref)
        s = np.take_along_axis(1 / (1 + np.exp(-z.astype(np.float64))), ref, 1)
        assert np.allclose(to_host(got[1]), s / s.sum(1, keepdims=True), rtol=1e-5)
        if stats:
            assert np.array_equal(to_host(got[2])[0], np.bincount(ref.reshape(-1), minlength=E))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k", [(70, 24, 3), (70, 96, 5), (45, 64, 20), (45, 200, 20), (20, 400, 24)])
def test_gradient_of_other_sizes(T, E, k, score, bf16):
    torch, fp8bs = require_gpu()
    z = _logits(T, E, T * E, bf16)
    seq = [0, T // 2, T]
    zd, sd = _dev(torch, z, bf16), to_dev(np.array(seq, np.int32))
    kw = dict(score=score, scale=1.5, alpha=0.7)
    idx, w, counts, tokens, loss = fp8bs.moe_route(zd, k, seq=sd, **kw)
    ri, rw, rc, rt, rl = route.route(z, k, seq=seq, **kw)
    assert np.array_equal(to_host(idx), ri) and np.array_equal(to_host(counts), rc) and np.allclose(to_host(loss), rl, rtol=2e-5)
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    got = to_host(fp8bs.moe_route_backward(zd, idx, to_dev(dw), seq=sd, counts=counts, tokens=tokens,
                                           dloss=to_dev(np.array([1.3], np.float32)), **kw))
    ref = route.backward(z, ri, dw, 1.3, seq=seq, **kw)
    tol = 2e-5 * np.abs(ref).max(axis=1, keepdims=True) + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 1e-30
    assert np.all(np.abs(got - ref) <= tol), np.abs(got - ref).max()
