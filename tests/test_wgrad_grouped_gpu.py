"""The experts' weight gradients against float64 products of the values that the codes stand for.

Tolerances are the GEMMs' (tests/_parity.py): 1e-5 of the terms' magnitude for float32, one BF16 ulp for BF16."""
import numpy as np
import pytest

import oracle
from oracle import train
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_host
from _parity import check_bf16, check_f32

pytestmark = pytest.mark.gpu


def _operand(width, R, seed, sigma=1.0, live=None):
    """Codes [width, R], scales [R/128, width] and the values; columns that are not live are zeros."""
    v = oracle.bf16_bits_to_f32(synth.normal_bf16((width, R), sigma, seed, 4, outliers=True)).copy()
    if live is not None:
        v[:, ~live] = 0.0
    q, s = oracle.quantize_act_1x128(v.astype(np.float32), pow2=True)
    return q, np.ascontiguousarray(s.T), oracle.dequantize_1x128(q, s).astype(np.float64)


def _run(offsets, N, K, R, out_dtype=None, accumulate=False, seed=0):
    torch, fp8bs = require_gpu()
    live = np.zeros(R, bool)
    for lo, hi in zip(offsets, offsets[1:]):
        live[lo:max(lo, hi - (37 if hi - lo > 64 else 0))] = True       # the last rows of a segment are padding
    a, sa, va = _operand(N, R, seed, 1e-3, live)
    b, sb, vb = _operand(K, R, seed + 1, 1.0, live)
    # what lies outside every segment is not read: not a number, scales that the product would refuse
    for lo, hi in [(0, offsets[0]), (offsets[-1], R)]:
        a[:, lo:hi], b[:, lo:hi] = 0x7F, 0x7F
        sa[lo // 128:hi // 128], sb[lo // 128:hi // 128] = 3.0, np.nan
    ref, mag = train.grouped_wgrad(va, vb, offsets)
    G = len(offsets) - 1
    out = None
    if accumulate:
        held = np.random.default_rng(7).standard_normal((G, N, K)).astype(np.float32)
        out = to_dev(held)
        ref, mag = ref + held, mag + np.abs(held)
    d = fp8bs.grouped_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(np.asarray(offsets, np.int32)), out_dtype, out,
                            accumulate)
    status = fp8bs.fp8bs_get_device_status()
    assert status == 0, status
    if out_dtype is None:
        check_f32(to_host(d), ref, mag, "dW")
    else:
        check_bf16(to_host(d), ref, mag, "dW")
    return d, ref


SHAPES = [([0, 128], 128, 128, 128), ([0, 256, 256, 896], 256, 384, 896), ([128, 384, 384, 384, 1664], 384, 640, 2048),
          ([0, 0, 0, 128, 128], 128, 256, 256), ([0, 1152, 1280], 1152, 256, 1280), ([0, 128, 256, 384, 512, 640], 1024, 1408, 640),
          ([0, 4096], 512, 256, 4096), ([0, 384, 1024, 1024, 1920, 3200], 1152, 1408, 3200), ([256, 768, 1408], 2304, 2176, 1536)]


@pytest.mark.parametrize("offsets,N,K,R", SHAPES)
def test_float32(offsets, N, K, R):
    d, ref = _run(offsets, N, K, R)
    for g in range(len(offsets) - 1):
        if offsets[g] == offsets[g + 1]:
            assert not to_host(d)[g].any()


@pytest.mark.parametrize("offsets,N,K,R", SHAPES)
def test_bf16(offsets, N, K, R):
    torch, _ = require_gpu()
    _run(offsets, N, K, R, torch.bfloat16)


@pytest.mark.parametrize("offsets,N,K,R", SHAPES)
def test_accumulate(offsets, N, K, R):
    _run(offsets, N, K, R, accumulate=True)


def test_one_expert_is_the_dense_product():
    """One segment: the dense Wgrad with row scales in the MMA, to float32's summation order."""
    torch, fp8bs = require_gpu()
    R, N, K = 1024, 256, 512
    a, sa, va = _operand(N, R, 3)
    b, sb, vb = _operand(K, R, 4)
    off = to_dev(np.array([0, R], np.int32))
    d = fp8bs.grouped_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), off)[0]
    dense = fp8bs.gemm(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), fp8bs.SCALE_ROW1x128, torch.float32, pow2=True)
    mag = np.abs(va) @ np.abs(vb).T
    assert np.all(np.abs(to_host(d).astype(np.float64) - to_host(dense)) <= 2e-5 * mag)


def test_many_experts():
    """512 experts (the most), most of them empty, and D's rows beyond 2^16."""
    G, N, K = 512, 256, 128
    counts = np.zeros(G, np.int64)
    counts[[0, 3, 77, 300, 511]] = [128, 256, 128, 384, 128]
    offsets = [0, *np.cumsum(counts).tolist()]
    _run(offsets, N, K, offsets[-1] + 128)


def test_invalid_offsets_and_scales_are_reported():
    torch, fp8bs = require_gpu()
    R, N, K = 512, 128, 128
    a, sa, _ = _operand(N, R, 5)
    b, sb, _ = _operand(K, R, 6)
    out = torch.full((2, N, K), 5.0, device="cuda:0")
    for bad in ([0, 100, 512], [0, 256, 128], [-128, 0, 128], [0, 128, 640]):
        fp8bs.grouped_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(np.array(bad, np.int32)), out=out)
        assert fp8bs.fp8bs_get_device_status() == 7
        assert bool((out == 5.0).all())
    good = to_dev(np.array([0, 128, 512], np.int32))
    for which in (0, 1):
        scales = [sa.copy(), sb.copy()]
        scales[which][1, 5] = 3.0
        fp8bs.grouped_wgrad(to_dev(a), to_dev(scales[0]), to_dev(b), to_dev(scales[1]), good, out=out)
        assert fp8bs.fp8bs_get_device_status() == 7
    fp8bs.grouped_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), good, out=out)
    assert fp8bs.fp8bs_get_device_status() == 0


def test_graph_with_other_segments():
    """Captured with one set of segments, replayed with another."""
    torch, fp8bs = require_gpu()
    R, N, K = 1280, 384, 256
    a, sa, va = _operand(N, R, 8)
    b, sb, vb = _operand(K, R, 9)
    args = [to_dev(v) for v in (a, sa, b, sb)]
    off = to_dev(np.array([0, 512, 512, 1280], np.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8bs.grouped_wgrad(*args, off)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            d = fp8bs.grouped_wgrad(*args, off)
    torch.cuda.synchronize()
    for offsets in ([128, 256, 1152, 1152], [0, 0, 0, 128]):
        off.copy_(torch.tensor(offsets, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_f32(to_host(d), *train.grouped_wgrad(va, vb, offsets), "dW")
    assert fp8bs.fp8bs_get_device_status() == 0
