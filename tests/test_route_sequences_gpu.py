"""The router's sequences: work that grows with their number and no faster, runs of empty ones, and
boundaries that break the rules, which are reported and harmless wherever they are."""
import numpy as np
import pytest

from oracle import route
from _gpu import require_gpu, to_dev, to_host
from test_route_gpu import _logits

pytestmark = pytest.mark.gpu


def _ms(torch, call):
    """The fastest of five, on the device."""
    call()
    best = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best.append(a.elapsed_time(b))
    return min(best)


@pytest.mark.parametrize("backward", [False, True])
def test_time_is_linear_in_the_sequences(backward):
    """From 16384 to 65535 sequences of the same tokens: 4 times the work if linear, 16 if quadratic; below 8."""
    torch, fp8bs = require_gpu()
    T, E, k = 65535, 64, 4
    z = to_dev(_logits(T, E, 1))
    ms = []
    for S in (16384, 65535):
        seq = to_dev(np.linspace(0, T, S + 1).astype(np.int32))
        idx, w, counts, tokens, loss = fp8bs.moe_route(z, k, seq=seq, alpha=0.1)
        if backward:
            ms.append(_ms(torch, lambda: fp8bs.moe_route_backward(z, idx, w, seq=seq, alpha=0.1, counts=counts, tokens=tokens,
                                                                  dloss=loss)))
        else:
            ms.append(_ms(torch, lambda: fp8bs.moe_route(z, k, seq=seq, alpha=0.1)))
    assert fp8bs.fp8bs_get_device_status() == 0
    assert ms[1] < 8 * ms[0], ms


@pytest.mark.parametrize("backward", [False, True])
def test_empty_sequences_are_passed_over_at_once(backward):
    """Two sequences of many hold all tokens: from 8192 to 65535 of them 8 times the work if linear (the empty
    rows of counts), 64 if quadratic; below 16.  Counts, tokens and loss are those of the two alone."""
    torch, fp8bs = require_gpu()
    T, E, k = 4096, 64, 4
    z = to_dev(_logits(T, E, 2))
    ms = []
    for S in (8192, 65535):
        bounds = np.full(S + 1, T // 2 + 3, np.int32)
        bounds[0], bounds[-1] = 0, T
        seq = to_dev(bounds)
        idx, w, counts, tokens, loss = fp8bs.moe_route(z, k, seq=seq, alpha=0.1)
        if backward:
            ms.append(_ms(torch, lambda: fp8bs.moe_route_backward(z, idx, w, seq=seq, alpha=0.1, counts=counts, tokens=tokens,
                                                                  dloss=loss)))
        else:
            ms.append(_ms(torch, lambda: fp8bs.moe_route(z, k, seq=seq, alpha=0.1)))
        two = fp8bs.moe_route(z, k, seq=to_dev(np.array([0, T // 2 + 3, T], np.int32)), alpha=0.1)
        assert torch.equal(two[2], counts[[0, -1]]) and torch.equal(two[3], tokens[[0, -1]])
        assert not counts[1:-1].any() and np.isclose(float(loss), float(two[4]) * 2 / S, rtol=2e-5)
    assert fp8bs.fp8bs_get_device_status() == 0
    assert ms[1] < 16 * ms[0], ms


@pytest.mark.parametrize("score", [0, 1])
def test_many_sequences_against_the_oracle(score):
    torch, fp8bs = require_gpu()
    T, E, k, S = 700, 20, 3, 500
    z = _logits(T, E, 5)
    seq = np.sort(np.random.default_rng(S).integers(0, T + 1, S - 1))
    seq = np.concatenate([[0], seq, [T]]).astype(np.int32)
    idx, w, counts, tokens, loss = fp8bs.moe_route(to_dev(z), k, score, seq=to_dev(seq), alpha=0.7)
    ri, rw, rc, rt, rl = route.route(z, k, score, seq=seq, alpha=0.7)
    assert np.array_equal(to_host(idx), ri) and np.array_equal(to_host(counts), rc) and np.array_equal(to_host(tokens), rt)
    assert np.allclose(to_host(loss), rl, rtol=2e-5)
    dw = np.random.default_rng(1).standard_normal((T, k)).astype(np.float32)
    dz = to_host(fp8bs.moe_route_backward(to_dev(z), idx, to_dev(dw), score, seq=to_dev(seq), alpha=0.7, counts=counts,
                                          tokens=tokens, dloss=to_dev(np.array([1.3], np.float32))))
    ref = route.backward(z, ri, dw, 1.3, score, seq=seq, alpha=0.7)
    assert np.all(np.abs(dz - ref) <= 2e-5 * np.abs(ref).max(axis=1, keepdims=True) + 1e-30)


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("bad", [{0: 1}, {0: -5}, {-1: 19999}, {-1: 20001}, {7: LOW}, {7: HIGH}, {300: 0}, {500: 20000},
                                 {999: HIGH, 1000: LOW}, {i: HIGH - i for i in range(1001)}, {i: LOW for i in range(1001)},
                                 {i: 0 for i in range(1001)}, {i: 20000 for i in range(1001)}])
def test_bad_boundaries_anywhere_are_reported(bad):
    """Bounds past the tokens, negative, out of order: one of them or all; outputs around stay as they were."""
    torch, fp8bs = require_gpu()
    T, E, k, S = 20000, 16, 2, 1000
    z = to_dev(_logits(T, E, 1))
    seq = np.linspace(0, T, S + 1).astype(np.int64)
    for i, v in bad.items():
        seq[i] = v
    sd = to_dev(seq.astype(np.int32))
    n = fp8bs.moe_route_workspace_bytes(T, E, S)
    ws = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda:0")
    counts = torch.full((S + 1, E), 77, dtype=torch.int32, device="cuda:0")
    idx = torch.full((T + 1, k), 77, dtype=torch.int32, device="cuda:0")
    w = torch.full((T + 1, k), 77.0, device="cuda:0")
    tokens = torch.full((S + 1,), 77, dtype=torch.int32, device="cuda:0")
    loss = torch.full((2,), 77.0, device="cuda:0")
    dz = torch.full((T + 1, E), 77.0, device="cuda:0")
    fp8bs.fp8bs_moe_route(z, fp8bs.IN_F32, T, E, E, 0, None, None, sd, S, k, 1, 1.0, 0.1, idx, w, counts, tokens, loss, ws, n)
    assert fp8bs.fp8bs_get_device_status() == 7
    counts[:S] = 1
    tokens[:S] = 20
    idx[:T] = 0
    w[:T] = 0.5
    fp8bs.fp8bs_moe_route_backward(z, fp8bs.IN_F32, T, E, E, 0, None, sd, S, k, 1, 1.0, 0.1, idx, counts, tokens, w, loss, dz, E)
    assert fp8bs.fp8bs_get_device_status() == 7 and fp8bs.fp8bs_get_device_status() == 0
    assert torch.all(ws[n:] == 0x5A) and torch.all(counts[S] == 77) and torch.all(idx[T] == 77) and torch.all(w[T] == 77)
    assert int(tokens[S]) == 77 and float(loss[1]) == 77 and torch.all(dz[T] == 77)
