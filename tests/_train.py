"""Comparisons shared by the GPU tests of the training operators."""
import numpy as np

import oracle
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import to_host

F32_HALF = 2.0 ** -24      # half a float32 step, relative
BF16_HALF = 2.0 ** -8      # half a BF16 step, relative
BF16_LEAST = 2.0 ** -134   # half the smallest BF16 step


def f32(bits):
    return oracle.bf16_bits_to_f32(bits)


def bits_of(t):
    """The bit patterns of a bfloat16 CUDA tensor."""
    import torch
    return t.detach().view(torch.int16).cpu().numpy().view(np.uint16)


def check_near(got, ref, mag, steps, half, what):
    """|got - ref| within `steps` float32 roundings of the magnitude and one rounding of the output."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    err = np.abs(got - ref)
    bound = steps * F32_HALF * mag + half * (np.abs(ref) + steps * F32_HALF * mag) + BF16_LEAST
    assert got.shape == ref.shape, what
    bad = ~(err <= bound)
    if np.any(bad):
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values off; first at {i}: got {got[i]!r}, exact {ref[i]!r}, "
                             f"bound {bound[i]!r}")


def check_codes(q, s, values_bits, pow2, what):
    """Codes and scales (kb-major) are the quantiser's of the BF16 values, bit for bit."""
    ref_q, ref_s = oracle.quantize_act_1x128(values_bits, pow2=pow2)
    assert np.array_equal(to_host(q), ref_q), f"{what}: codes"
    assert np.array_equal(to_host(s).T.view(np.uint32), ref_s.view(np.uint32)), f"{what}: scales"


def bf16_of(v):
    """Float32 values rounded to BF16 (bit patterns)."""
    return synth.f32_to_bf16_bits(np.asarray(v, np.float32))
