"""Infinities and NaN that reach the training operators, as where something before them overflowed: they are outside
the operators' contract, but do not come out as numbers, and rows and values that do not meet them keep their bits."""
import numpy as np
import pytest

from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev_bf16, to_host
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
