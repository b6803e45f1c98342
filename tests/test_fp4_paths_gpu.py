"""Paths of the 4-bit operators that other tests do not reach: products of several m-tiles whose CTAs share
K, grouped products on CTA pairs in both formats, every BF16 gate of the SwiGLU, every quotient of the block
scales.  Tolerances as in test_fp4_gpu.py."""
import numpy as np
import pytest

from oracle import fp4
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _parity import check_bf16, check_f32
from test_fp4_gpu import _check_quant, _f32, _operand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K", [(129, 264, 4160), (200, 520, 7168), (257, 136, 4096), (300, 128, 3904), (511, 72, 4032),
                                   (130, 4096, 4096)])
def test_gemm_of_several_tiles_sharing_k(M, N, K, fmt, f32):
    """More than one m-tile, few tiles, K long enough to be shared by the CTAs of a cluster; ragged last tiles."""
    torch, fp8bs = require_gpu()
    a, va = _operand(fp8bs, M, K, fmt, 1, outliers=True)
    b, vb = _operand(fp8bs, N, K, fmt, 2, 0.02)
    out = torch.full((M + 1, N), 3.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda:0")
    fp8bs.gemm_fp4(a, b, fmt, out=out[:M])
    assert fp8bs.fp8bs_get_device_status() == 0
    assert torch.all(out[M] == 3.0)
    (check_f32 if f32 else check_bf16)(to_host(out[:M]), *fp4.gemm(va, vb), f"{M}x{N}x{K} fmt {fmt}")


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("fmt", [0, 1])
def test_grouped_gemm_on_pairs_sampled(fmt, f32):
    """Rows enough for CTA pairs; odd numbers of row tiles, an empty group, N and K that end inside a tile and a stage."""
    torch, fp8bs = require_gpu()
    G, N, K = 6, 1288, 576
    offsets = np.concatenate([[0], np.cumsum([640, 1152, 0, 128, 2432, 896])]).astype(np.int32)
    a, va = _operand(fp8bs, int(offsets[-1]), K, fmt, 7, outliers=True)
    wbits = synth.normal_bf16((G, N, K), 0.02, 8, 5)
    b = fp8bs.quantize_fp4(to_dev_bf16(wbits), fmt)
    y = to_host(fp8bs.grouped_gemm_fp4(a, to_dev(offsets), b, fmt, out_dtype=torch.float32 if f32 else torch.bfloat16))
    assert fp8bs.fp8bs_get_device_status() == 0
    for g in range(G):
        rows = np.arange(offsets[g], offsets[g + 1], 37)
        Y, T = fp4.gemm(va[rows], fp4.values(*fp4.quantize(_f32(wbits[g]), fmt), fmt))
        (check_f32 if f32 else check_bf16)(y[rows], Y, T, f"group {g}")


@pytest.mark.parametrize("up", [1.0, -1.5703125, 2.0 ** 70, -2.0 ** -40])
def test_swiglu_of_every_gate(up):
    """Each finite BF16 gate alone in its row, so that the row scale holds all bits of BF16(silu(gate) * up):
    those of expf and the IEEE division."""
    torch, fp8bs = require_gpu()
    gates = np.concatenate([np.arange(0x0000, 0x7F80), np.arange(0x8000, 0xFF80)]).astype(np.uint16)
    M, I = len(gates), 64
    bits = np.zeros((M, 2 * I), np.uint16)
    at = np.arange(M) * 13 % I
    bits[np.arange(M), at] = gates
    bits[np.arange(M), I + at] = synth.f32_to_bf16_bits(np.array([up], np.float32))[0]
    h = to_dev_bf16(bits)
    gate, u = h[:, :I].float(), h[:, I:].float()
    half = torch.exp(0.5 * gate)
    v = (torch.where(gate < -64, gate * half * half, gate / (1.0 + torch.exp(-gate))) * u).to(torch.bfloat16)
    ok = torch.isfinite(v).all(dim=1)
    assert int(ok.sum()) >= (65280 if abs(up) <= 1 else 65280 - 70 * 128)   # 2^70 times gates from 2^58 up overflows
    got = fp8bs.swiglu_quantize_fp4(h[ok], 0)
    _check_quant(got, to_host(v[ok].float()).astype(np.float32), 0, f"every gate, up {up}")


def test_scales_of_every_quotient():
    """Block maxima of every BF16 mantissa in the 27 binades below row maxima of every mantissa."""
    torch, fp8bs = require_gpu()
    top = 0x4000 + np.arange(128)                                     # 2 .. 4
    below = (0x4000 + np.arange(128)[None, :] - 128 * np.arange(27)[:, None]).reshape(-1)
    bits = np.zeros((128, 64 + 16 * below.size), np.uint16)
    bits[:, 0] = top
    cols = 64 + 16 * np.arange(below.size) + np.arange(below.size) % 16
    bits[:, cols] = np.where(below[None, :] > top[:, None], top[:, None], below[None, :])
    _check_quant(fp8bs.quantize_fp4(to_dev_bf16(bits), 0), _f32(bits), 0, "every quotient")
