"""Infinities and NaN that reach the training operators, as where something before them overflowed: they are outside
the operators' contract, but do not come out as numbers, and rows and values that do not meet them keep their bits."""
import numpy as np
import pytest

from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _train import bf16_of, bits_of

pytestmark = pytest.mark.gpu
NAN, INF, NEG_INF = 0x7FC0, 0x7F80, 0xFF80


def _nan_codes(q):
    return (to_host(q) & 0x7F) == 0x7F


def _same_rows(a, b, rows):
    """The rows of outputs [M, ...] are bit for bit alike."""
    import torch
    for x, y in zip(a, b):
        assert torch.equal(x[rows].view(torch.uint8) if x.dtype == torch.bfloat16 else x[rows],
                           y[rows].view(torch.uint8) if y.dtype == torch.bfloat16 else y[rows])


@pytest.mark.parametrize("M,K", [(40, 128), (12, 2048), (7, 7168), (3, 16384)])
@pytest.mark.parametrize("pow2,residual", [(True, True), (True, False), (False, False)])
def test_norm(M, K, pow2, residual):
    torch, fp8bs = require_gpu()
    x, res = synth.normal_bf16((M, K), 1.0, 90, 4), synth.normal_bf16((M, K), 1.0, 91, 4)
    gain = to_dev(np.linspace(0.5, 1.5, K).astype(np.float32))

    def run():
        q, s, y, r, rstd = fp8bs.rmsnorm_quantize(to_dev_bf16(x), gain, to_dev_bf16(res) if residual else None, 1e-6, pow2, bf16=True)
        return q, s.t().contiguous(), y, r, rstd

    clean = run()
    x[1, K - 5] = NAN
    x[2, 3] = INF
    q, s, y, r, rstd = got = run()
    assert np.isnan(to_host(y)[1]).all() and np.isnan(to_host(rstd)[1]) and _nan_codes(q)[1].all()
    assert not np.isfinite(to_host(y)[2, 3]) and _nan_codes(q)[2, 3]
    _same_rows(got, clean, [i for i in range(M) if i not in (1, 2)])


@pytest.mark.parametrize("M,K", [(40, 128), (700, 2048), (5, 16384)])
def test_norm_gradient(M, K):
    """A NaN in dy reaches its row of dx and its column of the gain's gradient, and no other."""
    torch, fp8bs = require_gpu()
    r, dy, add = (synth.normal_bf16((M, K), 1.0, 92 + i, 4) for i in range(3))
    gain, rstd = to_dev(np.linspace(0.5, 1.5, K).astype(np.float32)), to_dev(np.full(M, 0.9, np.float32))

    def run():
        return fp8bs.rmsnorm_backward(to_dev_bf16(dy), to_dev_bf16(r), gain, rstd, to_dev_bf16(add))

    clean = run()
    dy[2, 9] = NAN
    add[4, 11] = INF
    dx, dgain = run()
    assert np.isnan(to_host(dx)[2]).all() and np.isposinf(to_host(dx)[4, 11])
    _same_rows((dx,), (clean[0],), [i for i in range(M) if i not in (2, 4)])
    assert np.isnan(to_host(dgain)[9])
    _same_rows((dgain,), (clean[1],), [i for i in range(K) if i != 9])


@pytest.mark.parametrize("M,I", [(6, 128), (300, 384), (700, 2048), (5, 4224)])
@pytest.mark.parametrize("pow2", [False, True])
def test_swiglu_gradient(M, I, pow2):
    """dgate = dv up s (1 + g s(-g)) and dup = dv g s term by term: dup of an infinite gate is infinite, where it is positive
    and dv is not zero; 0 times an infinity is NaN."""
    torch, fp8bs = require_gpu()
    h, dv = synth.normal_bf16((M, 2 * I), 2.0, 95, 4), synth.normal_bf16((M, I), 1.0, 96, 4)

    def run():
        q, s, dh = fp8bs.swiglu_backward_quantize(to_dev_bf16(h), to_dev_bf16(dv), None, pow2, bf16=True)
        return q, s.t().contiguous(), dh

    dv[0] = bf16_of(np.where(np.arange(I) % 2, -2.0, 0.5).astype(np.float32))
    clean = run()
    h[0, 1], h[0, 2], h[0, 4], h[0, 7], dv[0, 7] = INF, INF, NEG_INF, INF, 0
    h[1, 5], h[1, 6] = NAN, 0xFFC0                      # gates
    h[2, I + 3], dv[2, 70] = NAN, NAN
    h[3, I + 9], dv[3, 80] = INF, NEG_INF
    q, _, dh = got = run()
    v, want = to_host(dh), to_host(clean[2])
    assert np.isneginf(v[0, I + 1]) and np.isposinf(v[0, I + 2]) and np.isnan(v[0, [1, 2, 4, 7, I + 4, I + 7]]).all()
    assert np.isnan(v[1, [5, 6, I + 5, I + 6]]).all()
    assert np.isnan(v[2, [3, 70, I + 70]]).all() and v[2, I + 3] == want[2, I + 3]
    assert np.isinf(v[3, 9]) and np.isinf(v[3, [80, I + 80]]).all()
    assert _nan_codes(q)[~np.isfinite(v)].all()
    touched = {0: [1, 2, 4, 7], 1: [5, 6], 2: [3, 70], 3: [9, 80]}
    keep = np.ones((M, 2 * I), bool)
    for row, cols in touched.items():
        keep[row, cols] = keep[row, [I + c for c in cols]] = False
    assert np.array_equal(bits_of(dh)[keep], bits_of(clean[2])[keep])
    _same_rows(got, clean, [i for i in range(M) if i > 3])


@pytest.mark.parametrize("T", [9, 400])
@pytest.mark.parametrize("pow2", [False, True])
def test_combine_gradient(T, pow2):
    """An infinity of dout times a weight of zero is NaN, and shows in the codes of its group."""
    torch, fp8bs = require_gpu()
    k, N = 2, 384
    rows = 2 * T
    row_of, row_token = np.arange(rows, dtype=np.int32).reshape(T, k), np.repeat(np.arange(T, dtype=np.int32), k)
    dout, y = synth.normal_bf16((T, N), 1.0, 97, 4), synth.normal_bf16((rows, N), 1.0, 98, 4)
    w = np.full((T, k), 0.5, np.float32)
    w[[1, 2], 0] = 0.0

    def run():
        q, s, dy, dw = fp8bs.moe_combine_backward(to_dev_bf16(dout), to_dev_bf16(y), to_dev(row_of), to_dev(row_token), to_dev(w), pow2,
                                                  bf16=True)
        return q, s.t().contiguous(), dy, dw.reshape(rows)

    clean = run()
    dout[1, 200], dout[2, 5], dout[3, 300] = INF, NAN, NEG_INF
    q, _, dy, dw = got = run()
    v, codes = to_host(dy), _nan_codes(q)
    assert np.isnan(v[2, 200]) and np.isposinf(v[3, 200]) and np.isnan(v[4:6, 5]).all() and np.isneginf(v[6:8, 300]).all()
    assert codes[2:4, 200].all() and codes[5, 5] and codes[6:8, 300].all()
    assert not np.isfinite(to_host(dw)[2:8]).any()
    _same_rows(got, clean, [i for i in range(rows) if not 2 <= i < 8])
    _same_rows((q[:, :128], dy[:, :128]), (clean[0][:, :128], clean[2][:, :128]), [2, 3, 6, 7])    # groups beside theirs
