"""Gradient of the SwiGLU with 8-bit output, against float64.

Roundings: dup = dv (gate sigma) takes the exponential (2 steps of float32, CUDA's bound for expf), 1 + e, the
reciprocal (1 step), e c and two products: below 12 halves.  dgate takes as many and gate sigma(-gate) + 1, two
products more: 24 halves of its magnitude, with 1 + |gate| sigma(-gate) in the place of 1 + gate sigma(-gate).
Products of dv and up below float32's normal numbers lose 2^-150 at most, below BF16's least step."""
import numpy as np
import pytest

from oracle import train
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _train import BF16_HALF, bf16_of, bits_of, check_codes, check_near, f32

pytestmark = pytest.mark.gpu


def _check(h, dv, I, pow2=True, live=None):
    torch, fp8bs = require_gpu()
    q, s, dh = fp8bs.swiglu_backward_quantize(to_dev_bf16(h), to_dev_bf16(dv), None if live is None else to_dev(live), pow2, bf16=True)
    ref, mag = train.swiglu_backward(f32(h), f32(dv), I)
    if live is not None:
        ref[live < 0] = mag[live < 0] = 0.0
    check_near(to_host(dh), ref, mag, 24, BF16_HALF, "dh")
    check_codes(q, s, bits_of(dh), pow2, "dh")
    again = fp8bs.swiglu_backward_quantize(to_dev_bf16(h), to_dev_bf16(dv), None if live is None else to_dev(live), pow2)
    assert again[2] is None and torch.equal(again[0], q) and torch.equal(again[1], s)
    return dh


@pytest.mark.parametrize("M,I", [(1, 128), (1, 2048), (3, 256), (127, 384), (128, 128), (257, 2048), (65, 4096), (5, 1408)])
@pytest.mark.parametrize("pow2", [False, True])
def test_gradient(M, I, pow2):
    h, dv = synth.normal_bf16((M, 2 * I), 2.0, 50 + M, 5), synth.normal_bf16((M, I), 1e-3, 51 + M, 4, outliers=True)
    _check(h, dv, I, pow2)


def test_every_gate():
    """All finite BF16 gates from -170 up (e^gate is a float32 number above that), with ordinary and with large factors;
    below -170 the gradient of ordinary factors is below BF16's least value or zero."""
    g = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    g = g[np.isfinite(f32(g))]
    near = g[f32(g) >= -170]
    I = 128
    for up, dv in ((1.25, -0.75), (-3e20, 2e5), (3e-3, 1e-20)):
        n = -(-near.size // I)
        gate = np.resize(near, n * I).reshape(n, I)
        if up < 0:
            gate = np.where(np.abs(f32(gate)) < 1e9, gate, 0).astype(np.uint16)    # products of all three stay finite
        h = np.concatenate([gate, np.full((n, I), bf16_of(up))], axis=1)
        _check(h, np.full((n, I), bf16_of(dv)), I)
    far = g[f32(g) < -170]
    n = -(-far.size // I)
    h = np.concatenate([np.resize(far, n * I).reshape(n, I), np.full((n, I), bf16_of(2.0))], axis=1)
    dh = _check(h, np.full((n, I), bf16_of(0.5)), I)
    assert float(dh.float().abs().max()) < 2.0 ** -126


def test_zeros_and_signs():
    I = 128
    h = np.zeros((4, 2 * I), np.uint16)
    h[1] = 0x8000
    h[2, :I], h[2, I:] = bf16_of(1.0), 0
    h[3, :I], h[3, I:] = 0, bf16_of(1.0)
    dv = np.full((4, I), bf16_of(1.0))
    _check(h, dv, I)
    _check(h, np.zeros_like(dv), I, False)


def test_rows_without_a_token_are_not_read():
    """Padding holds whatever was there: NaN in h and dv of such rows leaves no trace."""
    M, I = 300, 256
    h, dv = synth.normal_bf16((M, 2 * I), 2.0, 60, 5), synth.normal_bf16((M, I), 1e-3, 61, 4)
    live = np.where(np.random.default_rng(0).random(M) < 0.4, -1, 7).astype(np.int32)
    torch, fp8bs = require_gpu()
    clean = fp8bs.swiglu_backward_quantize(to_dev_bf16(np.where(live[:, None] < 0, 0, h).astype(np.uint16)),
                                           to_dev_bf16(dv), to_dev(live), True, bf16=True)
    hn, dn = h.copy(), dv.copy()
    hn[live < 0], dn[live < 0] = 0x7FC0, 0x7FC0
    dirty = fp8bs.swiglu_backward_quantize(to_dev_bf16(hn), to_dev_bf16(dn), to_dev(live), True, bf16=True)
    for a, b in zip(clean, dirty):
        assert torch.equal(a.view(torch.uint8) if a.dtype == torch.bfloat16 else a, b.view(torch.uint8) if b.dtype == torch.bfloat16 else b)
    assert not to_host(dirty[0])[live < 0].any() and not to_host(dirty[1]).T[live < 0].any()
    _check(h, dv, I, True, live)
    _check(h, dv, I, True, np.full(M, -1, np.int32))


def test_strided_inputs():
    torch, fp8bs = require_gpu()
    M, I = 130, 384
    h, dv = to_dev_bf16(synth.normal_bf16((M, 2 * I + 64), 2.0, 62, 5))[:, :2 * I], to_dev_bf16(synth.normal_bf16((M, I + 8), 1.0, 63, 4))[:, :I]
    for a, b in zip(fp8bs.swiglu_backward_quantize(h, dv, pow2=True, bf16=True),
                    fp8bs.swiglu_backward_quantize(h.contiguous(), dv.contiguous(), pow2=True, bf16=True)):
        assert torch.equal(a, b)


def test_many_rows_sampled():
    """The experts' rows of 8192 tokens, inner size 2048; rows sampled for the float64 form."""
    torch, fp8bs = require_gpu()
    M, I = 67712, 2048
    torch.manual_seed(0)
    h = torch.randn((M, 2 * I), device="cuda:0").mul_(2).bfloat16()
    dv = torch.randn((M, I), device="cuda:0").mul_(1e-3).bfloat16()
    q, s, dh = fp8bs.swiglu_backward_quantize(h, dv, pow2=True, bf16=True)
    rows = torch.arange(0, M, 997, device="cuda:0")
    ref, mag = train.swiglu_backward(to_host(h[rows]), to_host(dv[rows]), I)
    check_near(to_host(dh[rows]), ref, mag, 24, BF16_HALF, "dh")
    check_codes(q[rows], s[:, rows].contiguous(), bits_of(dh[rows]), True, "dh")


@pytest.mark.parametrize("M,I,share", [(3000, 128, 1e-3), (2500, 1408, 1e-4), (1500, 4224, 1e-5), (700, 2048, 0.5), (1300, 384, 1e-3)])
def test_gates_far_below_here_and_there(M, I, share):
    """Gates below -64 in some rows, and in rows without a token, change no bit of the others."""
    torch, fp8bs = require_gpu()
    rng = np.random.default_rng(M)
    h, dv = synth.normal_bf16((M, 2 * I), 2.0, 64, 5), synth.normal_bf16((M, I), 1.0, 65, 4)
    live = np.where(rng.random(M) < 0.1, -1, 0).astype(np.int32)
    far = np.zeros((M, 2 * I), bool)
    far[:, :I] = rng.random((M, I)) < share
    far[0, 0] = far[-1, I - 1] = True
    wild = h.copy()
    wild[far] = bf16_of(-np.exp(rng.uniform(np.log(64.5), np.log(150.0), int(far.sum()))).astype(np.float32))
    with_far = _check(wild, dv, I, bool(M % 2), live)
    _, _, without = fp8bs.swiglu_backward_quantize(to_dev_bf16(h), to_dev_bf16(dv), to_dev(live), True, bf16=True)
    both = np.concatenate([far[:, :I], far[:, :I]], axis=1)
    assert np.array_equal(bits_of(with_far)[~both], bits_of(without)[~both])
