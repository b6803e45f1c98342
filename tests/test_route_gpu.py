"""Router, balance loss, their gradient and the row layout on the GPU against
the oracle (float64, token by token).

The choice is compared exactly: with softmax scores it goes by the logits, and
the inputs of the biased choice keep their keys further apart than float32
rounding (checked).  Weights: relative 1e-5 (a sum of up to 1024 float32
exponentials, at most 1024 * 2^-24 = 6e-5 in the worst order, the pairwise
order here below 2^-24 * 40 = 2.4e-6, and a few ulp more).  Loss and gradients:
float32 sums of like size, relative 2e-5 of the sum of their terms' magnitudes,
which the largest gradient of a token bounds from below within a factor of E.
"""
import numpy as np
import pytest

from oracle import route
from _gpu import require_gpu, to_dev, to_host

pytestmark = pytest.mark.gpu


def _logits(T, E, seed, bf16=False):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((T, E)) * 1.5 + rng.standard_normal((1, E)) * 0.5).astype(np.float32)
    if bf16:
        z = (z.view(np.uint32) & 0xFFFF0000).view(np.float32)       # BF16 values, ties among them
    return z


def _dev(torch, z, bf16):
    t = to_dev(z)
    return t.to(torch.bfloat16) if bf16 else t


def _gaps_ok(z, bias, k):
    """Whether the biased keys of every token differ by more than float32 rounding can move them."""
    key = np.sort(1 / (1 + np.exp(-z.astype(np.float64))) + bias, axis=1)
    return np.diff(key, axis=1).min(axis=1) > 1e-6


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score,T,E,k", [(0, 1, 1, 1), (0, 1, 256, 8), (1, 1, 256, 8), (0, 7, 5, 5), (1, 33, 31, 4),
                                         (0, 50, 33, 8), (1, 65, 64, 6), (0, 40, 100, 2), (1, 30, 257, 8),
                                         (0, 20, 513, 32), (1, 9, 1024, 32)])
def test_route(score, T, E, k, bf16):
    torch, fp8bs = require_gpu()
    z = _logits(T, E, T + E, bf16)
    idx, w = fp8bs.moe_route(_dev(torch, z, bf16), k, score, normalize=T % 2 == 1, scale=2.5)
    ri, rw, *_ = route.route(z, k, score, normalize=T % 2 == 1, scale=2.5)
    assert np.array_equal(to_host(idx), ri)
    assert np.allclose(to_host(w), rw, rtol=1e-5, atol=0)


@pytest.mark.parametrize("T,E,k", [(60, 64, 6), (200, 256, 8), (31, 40, 3)])
def test_route_with_bias(T, E, k):
    torch, fp8bs = require_gpu()
    rng = np.random.default_rng(E)
    z = _logits(4 * T, E, E)
    bias = (np.round(rng.standard_normal(E) * 100) * 1e-3).astype(np.float32)
    z = z[_gaps_ok(z, bias, k)][:T]
    assert len(z) > T // 2
    idx, w = fp8bs.moe_route(to_dev(z), k, fp8bs.SCORE_SIGMOID, bias=to_dev(bias))
    ri, rw, *_ = route.route(z, k, 1, bias=bias.astype(np.float64))
    assert np.array_equal(to_host(idx), ri) and np.allclose(to_host(w), rw, rtol=1e-5, atol=0)


@pytest.mark.parametrize("score", [0, 1])
def test_route_masks_and_edge_values(score):
    """Rows with fewer eligible experts than k or none, NaN and -inf logits, the type's lowest value, ties,
    signed zeros, masked tokens full of NaN, a row stride."""
    torch, fp8bs = require_gpu()
    T, E, k, ld = 12, 40, 4, 45
    z = _logits(T, E, 3)
    z[0] = -np.inf
    z[1] = np.nan
    z[2, 3:] = -np.inf
    z[3, ::2] = np.nan
    z[4] = 0.0
    z[4, 1::2] = -0.0
    z[5] = np.finfo(np.float32).min
    z[6, 5:] = np.finfo(np.float32).min
    z[7] = 1.25
    z[8] = np.nan
    z[9, 39] = np.finfo(np.float32).max / 4
    z[10] = -60.0
    valid = np.ones(T, np.uint8)
    valid[8] = valid[11] = 0
    wide = np.full((T, ld), 1e9, np.float32)
    wide[:, :E] = z
    for stats in (False, True):
        got = fp8bs.moe_route(to_dev(wide)[:, :E], k, score, valid=to_dev(valid), alpha=0.5 if stats else None)
        ref = route.route(z, k, score, valid=valid, alpha=0.5)
        assert np.array_equal(to_host(got[0]), ref[0])
        assert np.allclose(to_host(got[1]), ref[1], rtol=1e-5, atol=1e-30)
        if stats:
            assert np.array_equal(to_host(got[2]), ref[2]) and np.array_equal(to_host(got[3]), ref[3])
            assert np.allclose(to_host(got[4]), ref[4], rtol=2e-5)


SEQS = {"one": lambda T: None, "odd": lambda T: [0, 0, T // 3, T // 3, T // 3 + 1, T, T],
        "many": lambda T: [i * T // 23 for i in range(24)]}


@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("score,T,E,k,bf16", [(0, 130, 16, 2, False), (1, 600, 64, 6, False), (0, 77, 130, 8, True),
                                              (1, 1, 33, 3, False), (0, 41, 300, 5, False), (1, 25, 600, 7, True)])
def test_balance_loss_and_gradient(score, T, E, k, bf16, seqs):
    torch, fp8bs = require_gpu()
    z = _logits(T, E, T * E, bf16)
    rng = np.random.default_rng(T)
    valid = (rng.random(T) > 0.1).astype(np.uint8)
    z[rng.random((T, E)) < 0.02] = -np.inf
    if T > 30:
        z[17] = -np.inf
    seq = SEQS[seqs](T)
    dseq = None if seq is None else to_dev(np.array(seq, np.int32))
    zd, vd = _dev(torch, z, bf16), to_dev(valid)
    kw = dict(score=score, normalize=True, scale=2.5, alpha=0.7)
    idx, w, counts, tokens, loss = fp8bs.moe_route(zd, k, valid=vd, seq=dseq, **kw)
    ri, rw, rc, rt, rl = route.route(z, k, valid=valid, seq=seq, **kw)
    assert np.array_equal(to_host(idx), ri) and np.allclose(to_host(w), rw, rtol=1e-5, atol=1e-30)
    assert np.array_equal(to_host(counts), rc) and np.array_equal(to_host(tokens), rt)
    assert np.allclose(to_host(loss), rl, rtol=2e-5)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dw[ri < 0] = np.nan                                       # slots without an expert are not read
    dl = np.array([1.3], np.float32)
    for normalize, with_loss in ((True, True), (False, True), (True, False)):
        kw2 = dict(kw, normalize=normalize)
        got = fp8bs.moe_route_backward(zd, idx, to_dev(dw), valid=vd, seq=dseq, counts=counts if with_loss else None,
                                       tokens=tokens if with_loss else None, dloss=to_dev(dl) if with_loss else None, **kw2)
        ref = route.backward(z, ri, np.nan_to_num(dw), 1.3 if with_loss else 0.0, valid=valid, seq=seq, **kw2)
        got = to_host(got).astype(np.float64)
        big = np.abs(ref).max(axis=1, keepdims=True)
        tol = 2e-5 * big + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 1e-30
        assert np.all(np.abs(got - ref) <= tol), np.abs(got - ref).max()
        assert np.all(got[valid == 0] == 0) and np.all(got[~np.isfinite(z)] == 0)


def test_statistics_repeat_bit_for_bit_on_another_stream():
    torch, fp8bs = require_gpu()
    z, seq = to_dev(_logits(5000, 96, 1)), to_dev(np.array([0, 1700, 5000], np.int32))
    first = fp8bs.moe_route(z, 4, 0, seq=seq, alpha=0.01)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = fp8bs.moe_route(z, 4, 0, seq=seq, alpha=0.01)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("seq", [[0, 40, 99], [1, 40, 100], [0, 60, 40, 100], [0, 40, 101]])
def test_bad_sequences_are_refused(seq):
    torch, fp8bs = require_gpu()
    z, s = to_dev(_logits(100, 16, 1)), to_dev(np.array(seq, np.int32))
    idx, w, counts, tokens, loss = fp8bs.moe_route(z, 2, 0, seq=s, alpha=0.1)
    assert fp8bs.fp8bs_get_device_status() == 7
    fp8bs.moe_route_backward(z, torch.zeros_like(idx), w, seq=s, alpha=0.1)
    assert fp8bs.fp8bs_get_device_status() == 7 and fp8bs.fp8bs_get_device_status() == 0


def test_no_tokens():
    torch, fp8bs = require_gpu()
    z = torch.empty((0, 16), device="cuda:0")
    idx, w, counts, tokens, loss = fp8bs.moe_route(z, 2, 0, alpha=0.1)
    assert not counts.any() and not tokens.any() and float(loss) == 0.0
    offsets, row_token, row_of = fp8bs.moe_layout(idx, 16)
    assert not offsets.any() and row_token.numel() == 0


@pytest.mark.parametrize("T,k,E", [(1, 8, 256), (1, 1, 1), (5, 3, 4), (300, 8, 32), (255, 8, 1000), (700, 6, 64),
                                   (3000, 8, 96), (4100, 4, 1024)])
def test_layout(T, k, E):
    torch, fp8bs = require_gpu()
    rng = np.random.default_rng(T)
    p = (np.arange(E) + 1.0) ** -1.1
    idx = rng.choice(E, (T, k), p=p / p.sum()).astype(np.int32)     # repeats within a token too
    idx[rng.random((T, k)) < 0.05] = -1
    idx[rng.random((T, k)) < 0.02] = E                              # out of range: no row
    offsets, row_token, row_of = fp8bs.moe_layout(to_dev(idx), E)
    ro, rt, rr = route_layout(idx, E, row_token.numel())
    assert np.array_equal(to_host(offsets), ro)
    assert np.array_equal(to_host(row_token), rt) and np.array_equal(to_host(row_of), rr)


def route_layout(idx, E, rows):
    """route.layout in index arithmetic (the oracle's loops take minutes here); pinned against it."""
    T, k = idx.shape
    flat = idx.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")[:ok.sum()]
    counts = np.bincount(flat[ok], minlength=E)
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    first = np.cumsum(counts) - counts
    row = offsets[flat[order]] + np.arange(len(order)) - first[flat[order]]
    row_token, row_of = np.full(rows, -1), np.full(T * k, -1)
    row_token[row], row_of[order] = order // k, row
    return offsets, row_token, row_of.reshape(T, k)


def test_layout_arithmetic_is_the_oracles():
    idx = np.random.default_rng(0).integers(-1, 6, (40, 3))
    for a, b in zip(route_layout(idx, 5, 1024), route.layout(idx, 5, 1024)):
        assert np.array_equal(a, b)
