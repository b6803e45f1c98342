"""The training entry points refuse bad arguments before a GPU is touched."""
import pytest

import fp8_fine_grained_fp8bs_gb300 as fp8bs

FAKE = 1 << 20          # 16-byte aligned, never dereferenced: every call below fails its checks first
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    fp8bs.build()
    return fp8bs.load_library()


def _with(args, **changes):
    assert set(changes) <= set(args)
    return list({**args, **changes}.values())


NORM = dict(x=FAKE, M=128, K=256, ldx=256, residual=FAKE, ldr=256, gain=FAKE, kind=0, eps=1e-6, r=FAKE, y=None, q=FAKE, s=FAKE,
            mode=1, rstd=None, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(M=-1), INVALID), (dict(K=-8), INVALID), (dict(ldx=248), INVALID), (dict(ldr=248), INVALID), (dict(kind=2), INVALID),
    (dict(mode=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=1e-31), INVALID), (dict(x=None), INVALID), (dict(gain=None), INVALID),
    (dict(s=None), INVALID), (dict(q=None), INVALID), (dict(q=None, s=None), INVALID), (dict(r=None), INVALID),
    (dict(residual=None), INVALID), (dict(K=200), SHAPE), (dict(K=252, q=None, s=None, y=FAKE), SHAPE),
    (dict(K=16512, ldx=16512, ldr=16512), SHAPE), (dict(M=(1 << 31) + 1), SHAPE), (dict(x=FAKE + 2), ALIGN),
    (dict(residual=FAKE + 8), ALIGN), (dict(gain=FAKE + 4), ALIGN), (dict(r=FAKE + 2), ALIGN), (dict(y=FAKE + 4), ALIGN),
    (dict(q=FAKE + 8), ALIGN), (dict(s=FAKE + 2), ALIGN), (dict(rstd=FAKE + 1), ALIGN), (dict(ldx=260), ALIGN),
    (dict(ldr=257), ALIGN), (dict(M=0), OK), (dict(K=0), OK)])
def test_norm_refusals(lib, changes, status):
    assert lib.fp8bs_rmsnorm_quantize(*_with(NORM, **changes)) == status


BACK = dict(dy=FAKE, M=128, K=256, lddy=256, r=FAKE, ldr=256, gain=FAKE, kind=1, rstd=FAKE, dres=FAKE, lddres=256, dx=FAKE,
            dgain=FAKE, accumulate=0, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(M=-1), INVALID), (dict(lddy=248), INVALID), (dict(ldr=0), INVALID), (dict(lddres=255), INVALID), (dict(kind=-1), INVALID),
    (dict(dy=None), INVALID), (dict(r=None), INVALID), (dict(gain=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=100), INVALID), (dict(K=252), SHAPE),
    (dict(K=16392, lddy=16392, ldr=16392, lddres=16392), SHAPE), (dict(dy=FAKE + 2), ALIGN), (dict(dx=FAKE + 8), ALIGN),
    (dict(ws=FAKE + 8), ALIGN), (dict(dgain=FAKE + 2), ALIGN), (dict(lddy=260), ALIGN), (dict(lddres=260), ALIGN),
    (dict(K=0), OK), (dict(M=0, dgain=None), OK), (dict(M=0, accumulate=1), OK)])
def test_norm_gradient_refusals(lib, changes, status):
    assert lib.fp8bs_rmsnorm_backward(*_with(BACK, **changes)) == status


def test_norm_gradient_workspace(lib):
    f = lib.fp8bs_rmsnorm_backward_workspace_bytes
    assert [f(*a) for a in [(-1, 256), (1, 12), (1, 16392), (1 << 32, 256)]] == [-1] * 4
    assert f(0, 256) == 0 and 0 < f(1, 256) <= f(4096, 256) == f(1 << 20, 256)
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.rmsnorm_backward_workspace_bytes(1, 12)


SWIGLU = dict(h=FAKE, M=128, I=128, ldh=256, dv=FAKE, lddv=128, live=None, dh=None, q=FAKE, s=FAKE, mode=0, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(M=-1), INVALID), (dict(ldh=248), INVALID), (dict(lddv=120), INVALID), (dict(mode=-1), INVALID), (dict(h=None), INVALID),
    (dict(dv=None), INVALID), (dict(s=None), INVALID), (dict(q=None, s=None), INVALID), (dict(I=64), SHAPE),
    (dict(M=(1 << 31) + 1), SHAPE), (dict(h=FAKE + 2), ALIGN), (dict(dv=FAKE + 4), ALIGN), (dict(live=FAKE + 2), ALIGN),
    (dict(dh=FAKE + 8), ALIGN), (dict(ldh=260), ALIGN), (dict(lddv=132), ALIGN), (dict(M=0), OK), (dict(I=0), OK)])
def test_swiglu_gradient_refusals(lib, changes, status):
    assert lib.fp8bs_swiglu_backward_quantize(*_with(SWIGLU, **changes)) == status


COMBINE = dict(dout=FAKE, T=16, N=128, ldo=128, y=FAKE, rows=256, row_of=FAKE, row_token=FAKE, w=FAKE, k=2, dy=None, q=FAKE, s=FAKE,
               mode=1, dw=FAKE, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(T=-1), INVALID), (dict(rows=-1), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(mode=3), INVALID),
    (dict(ldo=120), INVALID), (dict(y=None), INVALID), (dict(q=None), INVALID), (dict(q=None, s=None), INVALID),
    (dict(row_token=None), INVALID), (dict(row_of=None), INVALID), (dict(w=None), INVALID), (dict(dout=None), INVALID),
    (dict(N=64), SHAPE), (dict(N=100, q=None, s=None, dy=FAKE, ldo=104), SHAPE), (dict(T=1 << 24), SHAPE),
    (dict(rows=(1 << 30) + 1), SHAPE), (dict(dout=FAKE + 2), ALIGN), (dict(y=FAKE + 8), ALIGN), (dict(row_of=FAKE + 2), ALIGN),
    (dict(w=FAKE + 1), ALIGN), (dict(dw=FAKE + 2), ALIGN), (dict(ldo=132), ALIGN), (dict(N=0), OK), (dict(T=0, rows=0), OK)])
def test_combine_gradient_refusals(lib, changes, status):
    assert lib.fp8bs_moe_combine_backward(*_with(COMBINE, **changes)) == status


DISPATCH = dict(d=FAKE, rows=256, N=128, row_of=FAKE, T=16, k=2, add=None, dx=FAKE, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(rows=-1), INVALID), (dict(k=65), INVALID), (dict(d=None), INVALID), (dict(row_of=None), INVALID), (dict(dx=None), INVALID),
    (dict(N=100), SHAPE), (dict(T=1 << 26), SHAPE), (dict(d=FAKE + 2), ALIGN), (dict(add=FAKE + 4), ALIGN),
    (dict(row_of=FAKE + 2), ALIGN), (dict(dx=FAKE + 8), ALIGN), (dict(T=0), OK), (dict(N=0), OK)])
def test_dispatch_gradient_refusals(lib, changes, status):
    assert lib.fp8bs_moe_dispatch_backward(*_with(DISPATCH, **changes)) == status


WGRAD = dict(a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, R=256, offsets=FAKE, G=2, d=FAKE, dt=0, N=128, K=128, accumulate=0, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(R=-128), INVALID), (dict(G=0), INVALID), (dict(G=513), INVALID), (dict(dt=2), INVALID), (dict(dt=1, accumulate=1), INVALID),
    (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(b=None), INVALID), (dict(sb=None), INVALID), (dict(offsets=None), INVALID),
    (dict(d=None), INVALID), (dict(R=200), SHAPE), (dict(N=64), SHAPE), (dict(K=192), SHAPE), (dict(R=1 << 31), SHAPE),
    (dict(N=1 << 24, G=128), SHAPE), (dict(N=1 << 20, K=1 << 24, G=2), SHAPE), (dict(a=FAKE + 8), ALIGN), (dict(sa=FAKE + 2), ALIGN),
    (dict(sb=FAKE + 4), ALIGN), (dict(offsets=FAKE + 1), ALIGN), (dict(d=FAKE + 8), ALIGN), (dict(N=0), OK), (dict(K=0), OK),
    (dict(R=0, accumulate=1), OK)])
def test_weight_gradient_refusals(lib, changes, status):
    assert lib.fp8bs_grouped_wgrad_pow2(*_with(WGRAD, **changes)) == status
