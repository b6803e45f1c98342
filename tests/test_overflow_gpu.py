"""Operators that quantise what they compute, where finite inputs give values beyond BF16's range: the codes
and scales are those of the quantiser on the BF16 values, infinities among them, so that an overflow shows."""
import numpy as np
import pytest

from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_dev_bf16
from _train import bf16_of, bits_of, f32

pytestmark = pytest.mark.gpu


def _as_unfused(q, s, values, pow2):
    """q and s against the quantiser of the BF16 values, some of them infinite, none NaN."""
    torch, fp8bs = require_gpu()
    v = values.float()
    assert bool(torch.isinf(v).any()) and bool(torch.isfinite(v).any()) and not bool(torch.isnan(v).any())
    q2, s2 = fp8bs.quantize_act(values, pow2=pow2)
    assert torch.equal(s.view(torch.int32), s2.view(torch.int32)), "scales"
    assert torch.equal(q, q2), "codes"
    # with power-of-two scales an infinity has the code of no number
    if pow2:
        assert bool(((q & 0x7F) == 0x7F)[torch.isinf(v)].all())


@pytest.mark.parametrize("M,K,residual", [(5, 256, False), (3, 7168, True), (3, 7168, False), (2, 16384, True), (9, 128, True)])
@pytest.mark.parametrize("pow2", [False, True])
def test_norm(M, K, residual, pow2):
    torch, fp8bs = require_gpu()
    x, res = (to_dev_bf16(synth.normal_bf16((M, K), 1.0, 70 + i, 4)) for i in range(2))
    gain = np.ones(K, np.float32)
    gain[3::31], gain[7::61] = 3e38, -2e38
    q, s, y, _, _ = fp8bs.rmsnorm_quantize(x, to_dev(gain), res if residual else None, 1e-6, pow2, bf16=True)
    _as_unfused(q, s, y, pow2)


@pytest.mark.parametrize("T", [9, 400])
@pytest.mark.parametrize("up", [10.0, 26.0])
@pytest.mark.parametrize("pow2", [False, True])
def test_combine_gradient(T, up, pow2):
    """Weights on both sides of 2^24, above which a scale is not divided out of them."""
    torch, fp8bs = require_gpu()
    k, N = 2, 384
    rows = 2 * T
    row_of = np.arange(rows, dtype=np.int32).reshape(T, k)
    dout = bf16_of(f32(synth.normal_bf16((T, N), 1.0, 72, 4)) * np.float32(2.0 ** (127.5 - up)))
    w = np.full((T, k), 2.0 ** up, np.float32)
    w[:, 1] *= -0.7
    q, s, dy, _ = fp8bs.moe_combine_backward(to_dev_bf16(dout), torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda:0"),
                                             to_dev(row_of), to_dev(np.repeat(np.arange(T, dtype=np.int32), k)), to_dev(w), pow2,
                                             bf16=True)
    with np.errstate(over="ignore"):
        want = bf16_of((f32(dout)[:, None, :] * w[:, :, None]).reshape(rows, N))
    assert np.array_equal(bits_of(dy), want)
    _as_unfused(q, s, dy, pow2)
    assert fp8bs.fp8bs_get_device_status() == 0


@pytest.mark.parametrize("M,I", [(3, 128), (700, 384), (5, 4224)])
@pytest.mark.parametrize("pow2", [False, True])
def test_swiglu_gradient(M, I, pow2):
    torch, fp8bs = require_gpu()
    h = synth.normal_bf16((M, 2 * I), 2.0, 73, 4)
    dv = synth.normal_bf16((M, I), 1.0, 74, 4)
    h[:, :I][:, 5::37] = bf16_of(2.0)
    h[:, I:][:, 5::37] = bf16_of(-3e30)
    dv[:, 5::37] = bf16_of(1e20)              # dgate overflows, dup does not
    h[:, :I][:, 90::129] = bf16_of(1e20)
    dv[:, 90::129] = bf16_of(-1e19)           # dup overflows
    h[:, I:][:, 90::129] = 0
    q, s, dh = fp8bs.swiglu_backward_quantize(to_dev_bf16(h), to_dev_bf16(dv), None, pow2, bf16=True)
    assert bool(torch.isinf(dh[:, 5].float()).all()) and bool(torch.isinf(dh[:, I + 90].float()).all())
    _as_unfused(q, s, dh, pow2)
