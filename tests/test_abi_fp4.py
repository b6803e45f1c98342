"""The 4-bit and routing entry points refuse bad arguments before a GPU is touched."""
import pytest

import fp8_fine_grained_fp8bs_gb300 as fp8bs

FAKE = 1 << 20          # 16-byte aligned, never dereferenced: every call below fails its checks first
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    fp8bs.build()
    return fp8bs.load_library()


def _with(args, **changes):
    out = dict(args)
    out.update(changes)
    return list(out.values())


QUANT = dict(x=FAKE, rows_in=128, K=128, ldx=128, rows=None, M=128, fmt=0, q=FAKE, sf=FAKE, g=FAKE, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(M=-1, rows_in=-1), INVALID), (dict(rows_in=127), INVALID), (dict(ldx=120), INVALID), (dict(fmt=2), INVALID),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(g=None), INVALID), (dict(sf=None), INVALID),
    (dict(K=96), SHAPE), (dict(M=1 << 31, rows_in=1 << 31), SHAPE), (dict(ldx=132), ALIGN), (dict(x=FAKE + 2), ALIGN),
    (dict(sf=FAKE + 8), ALIGN), (dict(rows=FAKE + 2), ALIGN), (dict(g=FAKE + 1), ALIGN), (dict(M=0, rows_in=0), OK)])
def test_quantize_refusals(lib, changes, status):
    assert lib.fp8bs_quantize_fp4(*_with(QUANT, **changes)) == status


def test_other_quantiser_refusals(lib):
    sw = dict(h=FAKE, M=128, I=128, ldh=256, live=None, fmt=0, q=FAKE, sf=FAKE, g=FAKE, stream=None)
    for changes, status in [(dict(ldh=248), INVALID), (dict(I=32), SHAPE), (dict(fmt=-1), INVALID), (dict(ldh=260), ALIGN),
                            (dict(g=None), INVALID), (dict(M=0), OK)]:
        assert lib.fp8bs_swiglu_quantize_fp4(*_with(sw, **changes)) == status, changes
    dq = dict(q=FAKE, sf=FAKE, g=FAKE, M=128, K=128, fmt=0, out=FAKE, dt=0, ldo=128, stream=None)
    for changes, status in [(dict(ldo=64), INVALID), (dict(dt=2), INVALID), (dict(K=100, ldo=100), SHAPE),
                            (dict(ldo=129), ALIGN), (dict(dt=1, ldo=132), ALIGN), (dict(out=None), INVALID), (dict(M=0), OK)]:
        assert lib.fp8bs_dequantize_fp4(*_with(dq, **changes)) == status, changes
    assert lib.fp8bs_fp4_scale_bytes(129, 192, 0) == 2 * 3 * 512
    assert lib.fp8bs_fp4_scale_bytes(129, 192, 1) == 2 * 2 * 512
    assert [lib.fp8bs_fp4_scale_bytes(*a) for a in [(-1, 64, 0), (1, 65, 0), (1, 64, 2)]] == [-1] * 3


GEMM = dict(a=FAKE, sfa=FAKE, ga=FAKE, b=FAKE, sfb=FAKE, gb=FAKE, fmt=0, d=FAKE, dt=0, M=128, N=128, K=128, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(M=-1), INVALID), (dict(fmt=3), INVALID), (dict(dt=2), INVALID), (dict(ga=None), INVALID), (dict(gb=None), INVALID),
    (dict(a=None), INVALID), (dict(sfb=None), INVALID), (dict(K=96), SHAPE), (dict(N=100), SHAPE), (dict(K=0), SHAPE),
    (dict(M=1 << 30, N=1 << 24), SHAPE), (dict(d=FAKE + 8), ALIGN), (dict(sfa=FAKE + 4), ALIGN), (dict(gb=FAKE + 4), ALIGN),
    (dict(M=0), OK), (dict(N=0), OK)])
def test_gemm_refusals(lib, changes, status):
    assert lib.fp8bs_gemm_fp4(*_with(GEMM, **changes)) == status
    grouped = dict(a=FAKE, sfa=FAKE, ga=FAKE, M=128, off=FAKE, G=2, b=FAKE, sfb=FAKE, gb=FAKE, fmt=0, d=FAKE, dt=0, N=128,
                   K=128, stream=None)
    assert lib.fp8bs_grouped_gemm_fp4(*_with(grouped, **changes)) == status
    assert lib.fp8bs_grouped_gemm_fp4(*_with(grouped, G=513)) == INVALID
    assert lib.fp8bs_grouped_gemm_fp4(*_with(grouped, off=None)) == INVALID


ROUTE = dict(z=FAKE, dt=0, T=10, E=16, ld=16, score=0, bias=None, valid=None, seq=None, S=1, k=2, norm=1, scale=1.0,
             alpha=0.0, idx=FAKE, w=FAKE, counts=None, tokens=None, loss=None, ws=None, n=0, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(dt=2), INVALID), (dict(score=2), INVALID), (dict(E=0, ld=1), INVALID), (dict(E=1025, ld=1025), INVALID),
    (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(E=64, ld=64, k=33), INVALID), (dict(ld=15), INVALID),
    (dict(S=2), INVALID), (dict(S=0, seq=FAKE), INVALID), (dict(bias=FAKE), INVALID), (dict(z=None), INVALID),
    (dict(idx=None), INVALID), (dict(loss=FAKE), INVALID), (dict(counts=FAKE, tokens=FAKE, loss=FAKE), INVALID),
    (dict(counts=FAKE, tokens=FAKE, loss=FAKE, ws=FAKE, n=8), INVALID), (dict(z=FAKE + 2), ALIGN), (dict(idx=FAKE + 1), ALIGN),
    (dict(dt=1, z=FAKE + 1), ALIGN), (dict(T=0), OK)])
def test_route_refusals(lib, changes, status):
    assert lib.fp8bs_moe_route(*_with(ROUTE, **changes)) == status


def test_route_backward_and_layout_refusals(lib):
    bw = dict(z=FAKE, dt=0, T=10, E=16, ld=16, score=0, valid=None, seq=None, S=1, k=2, norm=1, scale=1.0, alpha=0.0,
              idx=FAKE, counts=None, tokens=None, dw=FAKE, dloss=None, dz=FAKE, ldd=16, stream=None)
    for changes, status in [(dict(ldd=15), INVALID), (dict(dloss=FAKE), INVALID), (dict(dw=None), INVALID), (dict(S=3), INVALID),
                            (dict(dz=FAKE + 2), ALIGN), (dict(T=0), OK)]:
        assert lib.fp8bs_moe_route_backward(*_with(bw, **changes)) == status, changes
    rows = lib.fp8bs_moe_layout_rows(10, 2, 16)
    assert rows == (20 + 16 * 127 + 127) // 128 * 128
    lay = dict(idx=FAKE, T=10, k=2, E=16, off=FAKE, rt=FAKE, rows=rows, ro=FAKE, ws=FAKE, n=1 << 20, stream=None)
    for changes, status in [(dict(rows=rows - 1), SHAPE), (dict(T=1 << 24), SHAPE), (dict(k=65), INVALID), (dict(E=1025), INVALID),
                            (dict(ws=None), INVALID), (dict(off=None), INVALID), (dict(n=0), INVALID), (dict(ro=FAKE + 2), ALIGN)]:
        assert lib.fp8bs_moe_layout(*_with(lay, **changes)) == status, changes
    assert lib.fp8bs_moe_layout_rows(-1, 2, 16) == -1 and lib.fp8bs_moe_layout_workspace_bytes(10, 0, 16) == -1
    assert lib.fp8bs_moe_route_workspace_bytes(10, 0, 1) == -1
