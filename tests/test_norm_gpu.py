"""Root-mean-square norm with the residual's addition and 8-bit output, and its gradient, against float64.

Tolerances count roundings.  A row's sum of squares: a thread adds up to 32 terms, 5 steps over a warp's lanes and up
to 16 over warps, so below 64 float32 roundings of a positive sum, half as many on its root, then quotient,
addition, root and reciprocal: 40 in all.  y takes two products more: 44, and its rounding to BF16.  In the gradient
the mean of t r takes 64 roundings of its magnitude, rstd^3 and the products 12 more.  The gain's gradient adds a
thread's rows one after the other (M / 304 and one; fewer where up to 8 rows share a CTA and are added then), 304 / 32
parts a warp and 32 warps: below M / 304 + 1 + 8 + 10 + 32.
"""
import numpy as np
import pytest

from oracle import train
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _train import BF16_HALF, bf16_of, bits_of, check_codes, check_near, f32

pytestmark = pytest.mark.gpu
EPS = 1e-6
SIZES = [(1, 128), (1, 7168), (7, 128), (5, 256), (33, 512), (3, 640), (130, 2048), (19, 4096), (257, 7168), (2, 16384), (1000, 384)]


def _gain(K, kind, seed=0):
    g = (1 + 0.3 * np.random.default_rng(seed).standard_normal(K)).astype(np.float32)
    if kind == "f32":
        return to_dev(g), g
    b = bf16_of(g)
    return to_dev_bf16(b), f32(b)


def _rows(M, K, seed):
    return synth.normal_bf16((M, K), 1.0, seed, 1, outliers=True)


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("kind,pow2,residual", [("bf16", True, True), ("f32", False, False), ("f32", True, True), ("bf16", False, False)])
def test_norm(M, K, kind, pow2, residual):
    torch, fp8bs = require_gpu()
    x, res = _rows(M, K, 3), _rows(M, K, 4)
    gain, g = _gain(K, kind)
    q, s, y, r, rstd = fp8bs.rmsnorm_quantize(to_dev_bf16(x), gain, to_dev_bf16(res) if residual else None, EPS, pow2, bf16=True)
    rb = bf16_of(f32(x) + f32(res)) if residual else x
    assert np.array_equal(bits_of(r), rb)
    ref, ref_rstd = train.rmsnorm(f32(rb), g, EPS)
    check_near(to_host(rstd), ref_rstd, ref_rstd, 40, 0.0, "rstd")
    check_near(to_host(y), ref, np.abs(ref), 44, BF16_HALF, "y")
    check_codes(q, s, bits_of(y), pow2, "y")
    # the unfused quantiser gives the same bytes, and so does the call without the BF16 output
    q2, s2 = fp8bs.quantize_act(y, pow2=pow2)
    q3, s3, none, _, _ = fp8bs.rmsnorm_quantize(to_dev_bf16(x), gain, to_dev_bf16(res) if residual else None, EPS, pow2)
    assert none is None
    for a, b in ((q, q2), (s, s2), (q, q3), (s, s3)):
        assert torch.equal(a, b)
    assert fp8bs.fp8bs_get_device_status() == 0


@pytest.mark.parametrize("K", [8, 72, 200, 1000, 2056, 16376])
def test_bf16_output_alone_takes_any_multiple_of_8(K):
    torch, fp8bs = require_gpu()
    M = 13
    x = _rows(M, K, 5)
    gain, g = _gain(K, "f32")
    y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda:0")
    fp8bs.fp8bs_rmsnorm_quantize(to_dev_bf16(x), M, K, K, None, 0, gain, fp8bs.IN_F32, EPS, None, y, None, None)
    ref, _ = train.rmsnorm(f32(x), g, EPS)
    check_near(to_host(y), ref, np.abs(ref), 44, BF16_HALF, "y")


def test_rows_of_zeros_large_and_small_values():
    """A row of zeros gives zeros; values whose squares stay in float32's range keep their digits."""
    torch, fp8bs = require_gpu()
    K = 256
    x = f32(_rows(6, K, 6)).copy()
    x[0], x[1] = 0.0, -0.0
    x[2] *= np.float32(2.0 ** 54)
    x[3] *= np.float32(2.0 ** -70)
    x[4, 1:] = 0.0
    xb = bf16_of(x)
    gain, g = _gain(K, "bf16")
    for eps in (1e-6, 1e-30, 1.0):
        q, s, y, _, rstd = fp8bs.rmsnorm_quantize(to_dev_bf16(xb), gain, None, eps, True, bf16=True)
        ref, ref_rstd = train.rmsnorm(f32(xb), g, eps)
        check_near(to_host(rstd), ref_rstd, ref_rstd, 40, 0.0, "rstd")
        check_near(to_host(y), ref, np.abs(ref), 44, BF16_HALF, "y")
        check_codes(q, s, bits_of(y), True, "y")
        assert not to_host(s).T[:2].any() and not to_host(q)[0].any()


def test_strides_and_in_place():
    """Wider leading dimensions, and the sum written over the residual or over x."""
    torch, fp8bs = require_gpu()
    M, K, wide = 37, 384, 400
    x, res = _rows(M, wide, 7), _rows(M, wide, 8)
    gain, _ = _gain(K, "bf16")
    xd, rd = to_dev_bf16(x)[:, :K], to_dev_bf16(res)[:, :K]
    ref = fp8bs.rmsnorm_quantize(xd.contiguous(), gain, rd.contiguous(), EPS, True, bf16=True)
    for a, b in zip(fp8bs.rmsnorm_quantize(xd, gain, rd, EPS, True, bf16=True), ref):
        assert torch.equal(a, b)
    for over in (0, 1):
        a, b = xd.contiguous(), rd.contiguous()
        q, s = torch.empty_like(ref[0]), torch.empty_like(ref[1])
        fp8bs.fp8bs_rmsnorm_quantize(a, M, K, K, b, K, gain, fp8bs.IN_BF16, EPS, (a, b)[over], None, q, s, fp8bs.SCALE_POW2)
        assert torch.equal((a, b)[over], ref[3]) and torch.equal(q, ref[0]) and torch.equal(s, ref[1])


def _gradient_steps(M):
    return M / 304 + 1 + 8 + 10 + 32


@pytest.mark.parametrize("M,K", SIZES + [(4099, 264), (2500, 7168), (9, 8), (65, 1000), (11, 16376)])
@pytest.mark.parametrize("kind,dres", [("bf16", True), ("f32", False)])
def test_gradient(M, K, kind, dres):
    torch, fp8bs = require_gpu()
    r, dy, add = _rows(M, K, 9), synth.normal_bf16((M, K), 1e-3, 10, 4), synth.normal_bf16((M, K), 1e-3, 11, 4)
    gain, g = _gain(K, kind)
    rstd = train.rmsnorm(f32(r), g, EPS)[1].astype(np.float32)
    dx, dgain = fp8bs.rmsnorm_backward(to_dev_bf16(dy), to_dev_bf16(r), gain, to_dev(rstd), to_dev_bf16(add) if dres else None)
    ref, mag, ref_g, mag_g = train.rmsnorm_backward(f32(dy), f32(r), g, rstd, f32(add) if dres else None)
    check_near(to_host(dx), ref, mag, 80, BF16_HALF, "dx")
    check_near(to_host(dgain), ref_g, mag_g, _gradient_steps(M), 0.0, "dgain")
    # the same bits again, and added to what is there
    again = fp8bs.rmsnorm_backward(to_dev_bf16(dy), to_dev_bf16(r), gain, to_dev(rstd), to_dev_bf16(add) if dres else None)
    assert torch.equal(dx, again[0]) and torch.equal(dgain, again[1])
    held = torch.full((K,), 0.5, device="cuda:0")
    _, same = fp8bs.rmsnorm_backward(to_dev_bf16(dy), to_dev_bf16(r), gain, to_dev(rstd), to_dev_bf16(add) if dres else None,
                                     dgain=held)
    assert same is held and torch.equal(held, dgain + 0.5)


@pytest.mark.parametrize("M,K", [(4864, 8), (5003, 128), (9001, 264), (4871, 512), (4865, 504), (1000, 1536), (911, 1536), (912, 1160)])
@pytest.mark.parametrize("kind,dres", [("bf16", True), ("f32", False)])
def test_gradient_of_many_short_rows(M, K, kind, dres):
    """More rows share a CTA there; up to 16 sums of a row's threads then stand in for as many of its rows."""
    test_gradient(M, K, kind, dres)


def test_gradient_in_place_strided_and_without_the_gain():
    torch, fp8bs = require_gpu()
    M, K, wide = 61, 512, 520
    r, dy, add = (to_dev_bf16(synth.normal_bf16((M, wide), 1.0, 12 + i, 4))[:, :K] for i in range(3))
    gain, _ = _gain(K, "bf16")
    _, _, _, _, rstd = fp8bs.rmsnorm_quantize(r, gain)
    ref, ref_g = fp8bs.rmsnorm_backward(dy.contiguous(), r.contiguous(), gain, rstd, add.contiguous())
    got, got_g = fp8bs.rmsnorm_backward(dy, r, gain, rstd, add)
    assert torch.equal(got, ref) and torch.equal(got_g, ref_g)
    for over in range(3):
        t = [v.contiguous() for v in (dy, r, add)]
        fp8bs.fp8bs_rmsnorm_backward(t[0], M, K, K, t[1], K, gain, fp8bs.IN_BF16, rstd, t[2], K, t[over], None, 0, None, 0)
        assert torch.equal(t[over], ref)


def test_gradient_of_no_rows():
    torch, fp8bs = require_gpu()
    K = 256
    gain, _ = _gain(K, "f32")
    dx, dgain = fp8bs.rmsnorm_backward(torch.empty((0, K), dtype=torch.bfloat16, device="cuda:0"),
                                       torch.empty((0, K), dtype=torch.bfloat16, device="cuda:0"), gain,
                                       torch.empty(0, device="cuda:0"))
    assert dx.shape == (0, K) and not dgain.any()
    q, s, y, r, rstd = fp8bs.rmsnorm_quantize(torch.empty((0, K), dtype=torch.bfloat16, device="cuda:0"), gain)
    assert q.shape == (0, K) and s.shape == (2, 0) and rstd.shape == (0,)


def test_gradient_against_differences():
    """The kernels' own derivative: <y, dy> of the BF16 output changes by <dx, v> along v.  Steps of 2^-3 over
    4096 values: y's roundings (2^-8 relative, random) sum to sqrt(n) 2^-8 |dy|, a step's quotient 8 times that,
    and the second-order part cancels in the central difference; both stay below a twentieth of the slope along
    dx itself."""
    torch, fp8bs = require_gpu()
    M, K, h = 8, 512, 2.0 ** -3
    r, dy = f32(_rows(M, K, 20)), f32(synth.normal_bf16((M, K), 1.0, 21, 4))
    gain, g = _gain(K, "f32")
    rstd = train.rmsnorm(r, g, EPS)[1].astype(np.float32)
    dx, _ = fp8bs.rmsnorm_backward(to_dev_bf16(bf16_of(dy)), to_dev_bf16(bf16_of(r)), gain, to_dev(rstd))
    v = f32(bf16_of(np.sign(to_host(dx)) * 1.0))

    def value(x):
        y = fp8bs.rmsnorm_quantize(to_dev_bf16(bf16_of(x)), gain, None, EPS, bf16=True)[2]
        return float((to_host(y) * dy).sum())

    up, down = f32(bf16_of(r + h * v)), f32(bf16_of(r - h * v))
    moved = float((to_host(dx) * (up - down)).sum())
    assert abs(value(up) - value(down) - moved) < 0.05 * abs(moved)


def test_graph_and_two_streams():
    """Captured once and replayed on other inputs; two calls at once with a workspace each."""
    torch, fp8bs = require_gpu()
    M, K = 300, 1024
    gain, _ = _gain(K, "bf16")
    first, second = ([to_dev_bf16(_rows(M, K, 30 + 4 * n + i)) for i in range(4)] for n in range(2))

    def step(x, res, dy, add):
        q, s, _, r, rstd = fp8bs.rmsnorm_quantize(x, gain, res, EPS, True)
        return (q, s, r, rstd, *fp8bs.rmsnorm_backward(dy, r, gain, rstd, add))

    want = [[t.clone() for t in step(*a)] for a in (first, second)]
    held = [t.clone() for t in first]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(*held)
    torch.cuda.synchronize()
    for n, inputs in enumerate((second, first, second)):
        for a, b in zip(held, inputs):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[(n + 1) % 2]))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a = step(*first)
        with torch.cuda.stream(other):
            b = step(*second)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, want[0])) and all(torch.equal(p, q) for p, q in zip(b, want[1]))
