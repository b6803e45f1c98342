"""SwiGLU's gradient where dv * up, or its product with a part of the sigmoid, leaves float32's range on the way
to a result that is in BF16's.

Roundings of such values: below -64 the base-2 exponential is within 2 units in the last place (CUDA's bound for
exp2f), 4 halves of a step, its argument two roundings of numbers below 1/2, the product with dv up (1 + gate) two
more: 8.  From -64 up e^-gate (4), 1 + e, the quotient and four operations, the product: 12.  All below the 24 of the
ordinary ones."""
import numpy as np
import pytest

from oracle import train
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev_bf16, to_host
from _train import BF16_HALF, bf16_of, bits_of, check_near, f32

pytestmark = pytest.mark.gpu
BF16_MAX = 2.0 ** 128 - 2.0 ** 120
I = 256


def _run(h, dv, pow2=True):
    torch, fp8bs = require_gpu()
    q, s, dh = fp8bs.swiglu_backward_quantize(to_dev_bf16(h), to_dev_bf16(dv), None, pow2, bf16=True)
    ref, mag = train.swiglu_backward(f32(h), f32(dv), I)
    got = to_host(dh)
    beyond = np.abs(ref) >= BF16_MAX + 2.0 ** 120      # a step beyond BF16's largest number
    near = ~beyond & (np.abs(ref) > BF16_MAX - 2.0 ** 120)
    assert np.array_equal(np.where(beyond, got, 0), np.where(beyond, np.copysign(np.inf, ref), 0))
    keep = ~beyond & ~near
    check_near(np.where(keep, got, 0), np.where(keep, ref, 0), np.where(keep, mag, 0), 24, BF16_HALF, "dh")
    q2, s2 = fp8bs.quantize_act(dh, pow2=pow2)
    assert torch.equal(q, q2) and torch.equal(s.view(torch.int32), s2.view(torch.int32))
    return dh, beyond


@pytest.mark.parametrize("up,dv", [(1e20, 1e20), (-1e20, 3e38), (3e38, 0.1), (1e32, -1e32), (3e38, 3e38), (2e25, 1e30),
                                   (1e30, 3e30)])
def test_large_factors_over_the_gates(up, dv):
    """Every BF16 gate from -300 to 8: the products overflow where the gradient does not."""
    g = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    g = g[np.isfinite(f32(g))]
    g = g[(f32(g) >= -300) & (f32(g) <= 8)]
    n = -(-g.size // I)
    h = np.concatenate([np.resize(g, n * I).reshape(n, I), np.full((n, I), bf16_of(up))], axis=1)
    _run(h, np.full((n, I), bf16_of(dv)))


@pytest.mark.parametrize("up,dv", [(3e38, 1e-30), (1e-35, 2e38), (1e-20, 1e-20), (1e38, 1e-38), (2e-38, -3e38)])
def test_unlike_factors_at_low_gates(up, dv):
    """A large and a small factor: neither the sigmoid's part with the small one nor the rest may vanish on the way."""
    g = bf16_of(-np.linspace(60.0, 200.0, 4 * I).astype(np.float32)).reshape(4, I)
    h = np.concatenate([g, np.full((4, I), bf16_of(up))], axis=1)
    _run(h, np.full((4, I), bf16_of(dv)))


@pytest.mark.parametrize("pow2", [False, True])
def test_a_few_among_ordinary_values(pow2):
    """The other values of the rows keep their bits."""
    torch, fp8bs = require_gpu()
    M = 1300
    h, dv = synth.normal_bf16((M, 2 * I), 2.0, 80, 5), synth.normal_bf16((M, I), 1e-3, 81, 4)
    _, _, before = fp8bs.swiglu_backward_quantize(to_dev_bf16(h), to_dev_bf16(dv), None, pow2, bf16=True)
    at = np.random.default_rng(1).random((M, I)) < 2e-3
    at[0, 0] = at[-1, -1] = True
    h[:, :I][at], h[:, I:][at], dv[at] = bf16_of(-60.0), bf16_of(1e20), bf16_of(1e20)
    dh, beyond = _run(h, dv, pow2)
    assert not beyond.any() and bool(torch.isfinite(dh.float()).all())
    both = np.concatenate([at, at], axis=1)
    assert np.array_equal(bits_of(dh)[~both], bits_of(before)[~both])
