"""4-bit quantisers, dequantiser and GEMMs on the GPU against the oracle.

Codes, scale bytes and row scales must match bit for bit (every step of the
definition is one float32 operation); dequantised values too.  GEMM outputs:
FP32 within 1e-5 * sum|terms| of the exact sum (FP32 accumulation), BF16
within one BF16 ulp of its rounding (tests/_parity.py).
"""
import numpy as np
import pytest

import oracle
from oracle import fp4
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _parity import assert_bytes_equal, check_bf16, check_f32

pytestmark = pytest.mark.gpu

FILL = 0x5A


def _check_quant(got, x, fmt, what):
    q, sf, g = got
    codes, sf_ref, g_ref = fp4.quantize(x, fmt)
    assert_bytes_equal(to_host(q), fp4.pack(codes), f"{what}: codes")
    assert_bytes_equal(to_host(sf), fp4.tile_scales(sf_ref, fmt), f"{what}: scales")
    if fmt == 0:
        assert_bytes_equal(to_host(g).view(np.uint32), g_ref.view(np.uint32), f"{what}: row scales")
    else:
        assert g is None


def _f32(bits):
    return oracle.bf16_bits_to_f32(bits).astype(np.float32)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,K", [(1, 64), (1, 7168), (3, 192), (127, 1024), (128, 1088), (129, 2112), (257, 4160),
                                 (33, 8192), (5, 8256), (2, 16384), (3, 16448), (2, 40000)])
def test_quantize(M, K, fmt):
    torch, fp8bs = require_gpu()
    bits = synth.normal_bf16((M, K), 1.0, M + K, 1, outliers=True)
    _check_quant(fp8bs.quantize_fp4(to_dev_bf16(bits), fmt), _f32(bits), fmt, f"{M}x{K}")


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_special_rows(fmt):
    """Zero and tiny rows, subnormals, the largest BF16, -0, exact ties, one outlier in a row of small values."""
    torch, fp8bs = require_gpu()
    K = 256
    x = np.zeros((14, K), np.float32)
    x[1] = -0.0
    x[2, :] = np.float32(2.0 ** -133)                       # the smallest BF16 subnormal
    x[3, ::3] = np.float32(-2.0 ** -126)
    x[4, 7] = np.float32(3.3895e38)
    x[5] = np.float32(-3.3895e38)
    x[6, :16] = [6, -6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25]
    x[6, 16:32] = x[6, :16] * 448
    x[7] = np.linspace(-6, 6, K)
    x[8, 0], x[8, 1:] = 1e4, 1e-3
    x[9] = np.float32(2.0 ** -100) * np.linspace(-1, 1, K)
    x[10] = np.exp2(np.arange(K) % 40 - 20)
    x[11] = 1.5 * np.exp2(np.arange(K) // 32 - 4)           # amax = 1.5 * 2^e: the last value at this power of two
    x[12] = np.float32(1.5078125) * np.exp2(np.arange(K) // 32 - 4)
    x[13, 100] = -2.0 ** 127
    bits = synth.f32_to_bf16_bits(x)
    _check_quant(fp8bs.quantize_fp4(to_dev_bf16(bits), fmt), _f32(bits), fmt, "special rows")


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_every_magnitude(fmt):
    """Every finite positive BF16 value beside each of several row maxima."""
    torch, fp8bs = require_gpu()
    v = np.arange(0, 0x7F80, dtype=np.uint16)                # 32640 = 510 * 64
    rows = []
    for top in (0x7F7F, 0x4000, 0x3F80, 0x3D81, 0x0080):
        b = np.minimum(v, top).astype(np.uint16)
        b[1::2] |= 0x8000
        rows.append(np.random.default_rng(top).permutation(b))
    bits = np.stack(rows)
    _check_quant(fp8bs.quantize_fp4(to_dev_bf16(bits), fmt), _f32(bits), fmt, "all magnitudes")


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_strided_gathered_and_in_bounds(fmt):
    """A column slice of a wider matrix, rows picked by a list with padding and
    out-of-range entries, on a stream of its own; bytes past the outputs stay."""
    torch, fp8bs = require_gpu()
    rows_in, K, ld, M = 50, 320, 456, 131
    wide = synth.normal_bf16((rows_in, ld), 1.0, 5, 1, outliers=True)
    rng = np.random.default_rng(6)
    rows = rng.integers(-2, rows_in + 2, M).astype(np.int32)
    x = _f32(wide[:, 8:8 + K])
    ref = np.where(((rows >= 0) & (rows < rows_in))[:, None], x[np.clip(rows, 0, rows_in - 1)], np.float32(0))
    n_sf = fp8bs.fp4_scale_bytes(M, K, fmt)
    xd, rd = to_dev_bf16(wide), to_dev(rows)
    q = torch.full((M * K // 2 + 64,), FILL, dtype=torch.uint8, device="cuda:0")
    sf = torch.full((n_sf + 64,), FILL, dtype=torch.uint8, device="cuda:0")
    g = torch.full((M + 8,), 7.0, dtype=torch.float32, device="cuda:0")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fp8bs.fp8bs_quantize_fp4(xd[:, 8:], rows_in, K, ld, rd, M, fmt, q, sf, g if fmt == 0 else None)
    stream.synchronize()
    assert torch.all(q[M * K // 2:] == FILL) and torch.all(sf[n_sf:] == FILL) and torch.all(g[M:] == 7.0)
    _check_quant((q[:M * K // 2].view(M, K // 2), sf[:n_sf], g[:M] if fmt == 0 else None), ref, fmt, "gathered")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,I", [(1, 64), (37, 2048), (130, 704), (3, 16448)])
def test_swiglu_quantize(M, I, fmt):
    """v = gate / (1 + e^-gate) * up: within half a BF16 ulp (rounding) and 2^-21 |v|
    (expf once or twice, and three IEEE operations, 4 ulp in all) of the exact value; the codes are v's."""
    torch, fp8bs = require_gpu()
    bits = synth.normal_bf16((M, 2 * I), 3.0, M, 1, outliers=True)
    bits[0, :8] = synth.f32_to_bf16_bits(np.array([0, -0.0, 90, -90, -120, 3e4, -3e4, 1e-30], np.float32))
    live = np.where(np.random.default_rng(M).random(M) < 0.2, -1, 5).astype(np.int32)
    live[0] = 0
    h = to_dev_bf16(bits)
    gate, up = h[:, :I].float(), h[:, I:].float()
    half = torch.exp(0.5 * gate)
    v = (torch.where(gate < -64, gate * half * half, gate / (1.0 + torch.exp(-gate))) * up).to(torch.bfloat16).float()
    exact = oracle.swiglu(bits, I)
    got = to_host(v).astype(np.float64)
    big = np.maximum(np.abs(exact), 2.0 ** -126)
    assert np.all(np.abs(got - exact) <= big * (2.0 ** -8 + 2.0 ** -21))
    out = fp8bs.swiglu_quantize_fp4(h, fmt, live=to_dev(live))
    _check_quant(out, np.where((live >= 0)[:, None], to_host(v), np.float32(0)).astype(np.float32), fmt, "swiglu")
    _check_quant(fp8bs.swiglu_quantize_fp4(h, fmt), to_host(v).astype(np.float32), fmt, "swiglu, every row live")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,K", [(1, 64), (130, 192), (7, 7168), (300, 1984)])
def test_dequantize_every_code(M, K, fmt):
    torch, fp8bs = require_gpu()
    rng = np.random.default_rng(M)
    codes = rng.integers(0, 16, (M, K)).astype(np.uint8)
    J = K // fp4.GROUP[fmt]
    sf = rng.integers(0, 255, (M, J)).astype(np.uint8)
    if fmt == 0:
        sf[(sf & 0x7F) == 0x7F] = 0x7E
    else:
        sf[:] = np.clip(sf, 3, 250)                              # float32 holds 6 * 2^(b - 127)
        sf[0, 0] = 0                                             # 2^-127, a float32 subnormal
    g = np.exp2(rng.integers(-20, 20, M)).astype(np.float32) * np.float32(1.37) if fmt == 0 else None
    args = to_dev(fp4.pack(codes)), to_dev(fp4.tile_scales(sf, fmt)), to_dev(g) if fmt == 0 else None
    ref = fp4.values(codes, sf, None, fmt).astype(np.float32)      # exact
    if fmt == 0:
        ref = ref * g[:, None]                                   # one float32 rounding
    f = fp8bs.dequantize_fp4(*args, fmt, out_dtype=torch.float32)
    assert np.array_equal(to_host(f), ref)
    b = fp8bs.dequantize_fp4(*args, fmt)
    assert np.array_equal(to_host(b), oracle.bf16_round(ref.astype(np.float64)))
    wide = torch.full((M, K + 8), 3.0, dtype=torch.float32, device="cuda:0")
    fp8bs.fp8bs_dequantize_fp4(*args, M, K, fmt, wide, fp8bs.OUT_F32, K + 8)
    assert np.array_equal(to_host(wide[:, :K]), ref) and torch.all(wide[:, K:] == 3.0)


def _operand(fp8bs, rows, K, fmt, seed, sigma=1.0, outliers=False):
    bits = synth.normal_bf16((rows, K), sigma, seed, 1, outliers=outliers)
    codes, sf, g = fp4.quantize(_f32(bits), fmt)
    return fp8bs.quantize_fp4(to_dev_bf16(bits), fmt), fp4.values(codes, sf, g, fmt)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K", [(1, 8, 64), (1, 136, 256), (1, 2048, 7168), (2, 520, 1984), (7, 7168, 512),
                                   (16, 256, 4160), (31, 264, 320), (64, 1000, 2048), (128, 128, 128), (129, 392, 704),
                                   (200, 2056, 1088), (333, 1032, 1984), (640, 512, 192), (1000, 4104, 448)])
def test_gemm(M, N, K, fmt, f32):
    torch, fp8bs = require_gpu()
    a, va = _operand(fp8bs, M, K, fmt, 1, outliers=True)
    b, vb = _operand(fp8bs, N, K, fmt, 2, 0.02)
    out = torch.full((M + 1, N), 3.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda:0")
    fp8bs.gemm_fp4(a, b, fmt, out=out[:M])
    torch.cuda.synchronize()
    assert fp8bs.fp8bs_get_device_status() == 0
    assert torch.all(out[M] == 3.0)
    Y, T = fp4.gemm(va, vb)
    (check_f32 if f32 else check_bf16)(to_host(out[:M]), Y, T, f"{M}x{N}x{K} fmt {fmt}")


@pytest.mark.parametrize("fmt", [0, 1])
def test_gemm_pair_tiles_sampled(fmt):
    """Enough tiles for the CTA pairs, ragged in M, N and K."""
    torch, fp8bs = require_gpu()
    M, N, K = 4737, 2312, 832
    a, va = _operand(fp8bs, M, K, fmt, 3, outliers=True)
    b, vb = _operand(fp8bs, N, K, fmt, 4, 0.02)
    y = fp8bs.gemm_fp4(a, b, fmt, out_dtype=torch.float32)
    assert fp8bs.fp8bs_get_device_status() == 0
    rows = np.unique(np.concatenate([np.arange(0, M, 61), [127, 128, 255, 256, 4607, 4608, M - 1]]))
    Y, T = fp4.gemm(va[rows], vb)
    check_f32(to_host(y[to_dev(rows)]), Y, T, "pair tiles")


@pytest.mark.parametrize("fmt", [0, 1])
def test_gemm_distinct_scales_reach_their_rows_and_columns(fmt):
    """Codes of one, a scale of its own for every block: a scale that lands on
    another row, column or block of K changes the sum."""
    torch, fp8bs = require_gpu()
    M, N, K = 200, 200, 384
    rng = np.random.default_rng(9)
    J = K // fp4.GROUP[fmt]

    def make(rows):
        codes = np.full((rows, K), 2, np.uint8)
        sf = rng.integers(0x30, 0x50, (rows, J)).astype(np.uint8) if fmt == 0 else rng.integers(120, 134, (rows, J)).astype(np.uint8)
        g = np.exp2(rng.integers(-3, 3, rows)).astype(np.float32) if fmt == 0 else None
        dev = to_dev(fp4.pack(codes)), to_dev(fp4.tile_scales(sf, fmt)), None if g is None else to_dev(g)
        return dev, fp4.values(codes, sf, g, fmt)

    (a, va), (b, vb) = make(M), make(N)
    y = fp8bs.gemm_fp4(a, b, fmt, out_dtype=torch.float32)
    Y, T = fp4.gemm(va, vb)
    check_f32(to_host(y), Y, T, "distinct scales")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("G,N,K,segments", [
    (1, 264, 192, [128]), (3, 136, 320, [0, 128, 0]), (4, 392, 1984, [256, 0, 128, 384]),
    (5, 1032, 448, [128, 128, 640, 0, 128]), (32, 256, 256, [128 * (i % 3) for i in range(32)])])
def test_grouped_gemm(G, N, K, segments, fmt):
    torch, fp8bs = require_gpu()
    offsets = np.concatenate([[0], np.cumsum(segments)]).astype(np.int32)
    M = int(offsets[-1]) + 70                                  # rows past the segments, not a multiple of 128
    a, va = _operand(fp8bs, M, K, fmt, 5, outliers=True)
    wbits = synth.normal_bf16((G, N, K), 0.02, 6, 5)
    b = fp8bs.quantize_fp4(to_dev_bf16(wbits), fmt)
    y = torch.full((M, N), 3.0, dtype=torch.float32, device="cuda:0")
    fp8bs.grouped_gemm_fp4(a, to_dev(offsets), b, fmt, out=y)
    assert fp8bs.fp8bs_get_device_status() == 0
    got = to_host(y)
    for g in range(G):
        lo, hi = offsets[g], offsets[g + 1]
        Y, T = fp4.gemm(va[lo:hi], fp4.values(*fp4.quantize(_f32(wbits[g]), fmt), fmt))
        check_f32(got[lo:hi], Y, T, f"group {g}")
    assert np.all(got[offsets[-1]:] == 3.0)


def test_grouped_gemm_large_sampled():
    """Enough rows for the CTA pairs, odd numbers of row tiles in the groups."""
    torch, fp8bs = require_gpu()
    G, N, K, fmt = 6, 1288, 576, 0
    offsets = np.concatenate([[0], np.cumsum([640, 1152, 0, 128, 2432, 896])]).astype(np.int32)
    a, va = _operand(fp8bs, int(offsets[-1]), K, fmt, 7, outliers=True)
    wbits = synth.normal_bf16((G, N, K), 0.02, 8, 5)
    b = fp8bs.quantize_fp4(to_dev_bf16(wbits), fmt)
    y = to_host(fp8bs.grouped_gemm_fp4(a, to_dev(offsets), b, fmt))
    assert fp8bs.fp8bs_get_device_status() == 0
    for g in range(G):
        rows = np.arange(offsets[g], offsets[g + 1], 37)
        Y, T = fp4.gemm(va[rows], fp4.values(*fp4.quantize(_f32(wbits[g]), fmt), fmt))
        check_bf16(y[rows], Y, T, f"group {g}")


@pytest.mark.parametrize("offsets", [[0, 100, 256], [0, 256, 128], [-128, 128, 256], [0, 128, 512]])
def test_grouped_gemm_refuses_bad_offsets(offsets):
    torch, fp8bs = require_gpu()
    a, _ = _operand(fp8bs, 256, 128, 1, 1)
    b = fp8bs.quantize_fp4(to_dev_bf16(synth.normal_bf16((2, 128, 128), 1.0, 2, 5)), 1)
    y = torch.full((256, 128), 3.0, dtype=torch.float32, device="cuda:0")
    fp8bs.grouped_gemm_fp4(a, to_dev(np.array(offsets, np.int32)), b, 1, out=y)
    assert fp8bs.fp8bs_get_device_status() == 7
    assert torch.all(y == 3.0) and fp8bs.fp8bs_get_device_status() == 0


def test_grouped_gemm_without_rows():
    torch, fp8bs = require_gpu()
    a, _ = _operand(fp8bs, 256, 128, 0, 1)
    b = fp8bs.quantize_fp4(to_dev_bf16(synth.normal_bf16((3, 136, 128), 1.0, 2, 5)), 0)
    y = torch.full((256, 136), 3.0, dtype=torch.bfloat16, device="cuda:0")
    for offsets in ([0, 0, 0, 0], [128, 128, 128, 128]):
        fp8bs.grouped_gemm_fp4(a, to_dev(np.array(offsets, np.int32)), b, 0, out=y)
    assert fp8bs.fp8bs_get_device_status() == 0 and torch.all(y == 3.0)


def test_gemm_repeats_bit_for_bit():
    torch, fp8bs = require_gpu()
    a, _ = _operand(fp8bs, 5, 7168, 0, 1)
    b, _ = _operand(fp8bs, 264, 7168, 0, 2)
    ys = [fp8bs.gemm_fp4(a, b, 0, out_dtype=torch.float32) for _ in range(3)]
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
