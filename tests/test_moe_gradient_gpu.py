"""Gradients of the MoE combine and dispatch, against the float64 forms.

dy is the float32 product w dout rounded to BF16, bit for bit.  dw: a lane
adds each piece's 4 pairs of products (one rounding each, fused) to one of four pairs of sums, N / 1024 pieces a sum, then
8 sums, 5 steps over lanes and, where warps share a slot, 8 more.  dx: a rounding per addend of a float32 sum, then BF16's."""
import numpy as np
import pytest

from oracle import route, train
from fp8_fine_grained_fp8bs_gb300 import synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _train import BF16_HALF, bf16_of, bits_of, check_codes, check_near, f32

pytestmark = pytest.mark.gpu


def _layout(T, E, k, seed, masked=0.1):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random(T) < masked] = -1
    rows = -(-(T * k + min(E, T * k) * 127) // 128) * 128
    offsets, row_token, row_of = route.layout(idx, E, rows)
    return np.asarray(row_token, np.int32), np.asarray(row_of, np.int32), rows


def _expected_dy(dout, row_of, w, rows):
    """BF16 bits of the float32 products, row by row."""
    dy = np.zeros((rows, dout.shape[1]), np.uint16)
    for t, j in zip(*np.nonzero((row_of >= 0) & (row_of < rows))):
        dy[row_of[t, j]] = bf16_of(f32(dout[t]) * np.float32(w[t, j]))
    return dy


def _dot_steps(N):
    return 4 * -(-N // 1024) + 8 + 5 + 8


@pytest.mark.parametrize("T,E,k,N", [(1, 8, 2, 128), (1, 8, 8, 7168), (3, 5, 1, 256), (37, 16, 4, 640), (200, 63, 6, 2048),
                                     (700, 32, 8, 384), (129, 64, 13, 128), (5, 64, 64, 256),
                                     (350, 8, 3, 128), (6, 8, 2, 8320), (3, 4, 2, 20480)])
@pytest.mark.parametrize("pow2", [False, True])
def test_combine_gradient(T, E, k, N, pow2):
    torch, fp8bs = require_gpu()
    row_token, row_of, rows = _layout(T, E, k, T)
    dout, y = synth.normal_bf16((T, N), 1e-3, 1, 4, outliers=True), synth.normal_bf16((rows, N), 1.0, 2, 1)
    w = (0.02 + np.random.default_rng(3).random((T, k))).astype(np.float32) * np.where(np.arange(k) % 3 == 1, -1, 1).astype(np.float32)
    args = (to_dev_bf16(dout), to_dev_bf16(y), to_dev(row_of), to_dev(row_token), to_dev(w), pow2)
    q, s, dy, dw = fp8bs.moe_combine_backward(*args, bf16=True)
    want = _expected_dy(dout, row_of, w, rows)
    got = bits_of(dy)
    assert np.array_equal(got, want)
    check_codes(q, s, want, pow2, "dy")
    _, ref, mag = train.combine_backward(f32(dout), f32(y), row_of, w, rows)
    check_near(to_host(dw), ref, mag, _dot_steps(N), 0.0, "dw")
    assert not to_host(dw)[row_of < 0].any()
    q2, s2, none, dw2 = fp8bs.moe_combine_backward(*args)
    assert none is None and torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(dw, dw2)
    assert fp8bs.fp8bs_get_device_status() == 0


def test_padding_rows_are_zeroed_and_others_kept():
    """Rows without a token become zeros whatever they held; a row whose token does not name it is left as it is."""
    torch, fp8bs = require_gpu()
    T, k, N, rows = 4, 2, 128, 256
    row_of = np.array([[0, 128], [1, -1], [rows, 129], [-1, -1]], np.int32)
    row_token = np.full(rows, -1, np.int32)
    row_token[[0, 1, 128, 129, 130]] = [0, 1, 0, 2, 3]        # token 3 does not name row 130
    dout, y = synth.normal_bf16((T, N), 1.0, 5, 4), synth.normal_bf16((rows, N), 1.0, 6, 1)
    w = np.arange(1, 9, dtype=np.float32).reshape(T, k)
    q = torch.full((rows, N), 0x55, dtype=torch.uint8, device="cuda:0")
    s = torch.full((1, rows), 7.0, device="cuda:0")
    dy = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device="cuda:0")
    dw = torch.full((T, k), 9.0, device="cuda:0")
    fp8bs.fp8bs_moe_combine_backward(to_dev_bf16(dout), T, N, N, to_dev_bf16(y), rows, to_dev(row_of), to_dev(row_token), to_dev(w),
                                     k, dy, q, s, fp8bs.SCALE_POW2, dw)
    assert fp8bs.fp8bs_get_device_status() == 0
    want = _expected_dy(dout, row_of, w, rows)
    keep = np.zeros(rows, bool)
    keep[130] = True
    assert np.array_equal(bits_of(dy)[~keep], want[~keep]) and np.all(to_host(dy)[130] == 3.0)
    assert np.all(to_host(q)[130] == 0x55) and to_host(s)[0, 130] == 7.0
    assert not to_host(q)[row_token < 0].any() and not to_host(s)[0, row_token < 0].any()
    _, ref, mag = train.combine_backward(f32(dout), f32(y), row_of, w, rows)
    check_near(to_host(dw), ref, mag, _dot_steps(N), 0.0, "dw")


def test_same_row_twice_and_rows_of_another_token():
    """A row that two slots name takes both weights; a row that row_token gives to another token is reported."""
    torch, fp8bs = require_gpu()
    T, k, N, rows = 3, 4, 256, 128
    row_of = np.array([[5, 7, 5, -1], [9, 10, 11, 12], [20, 9, 21, 22]], np.int32)
    row_token = np.full(rows, -1, np.int32)
    for t in (0, 1, 2):
        row_token[[r for r in row_of[t] if r >= 0 and not (t == 2 and r == 9)]] = t
    dout, y = synth.normal_bf16((T, N), 1.0, 7, 4), synth.normal_bf16((rows, N), 1.0, 8, 1)
    w = np.array([[1, 2, 4, 8], [0.5, 1, 2, 3], [1, 1, 2, 2]], np.float32)
    q, s, dy, dw = fp8bs.moe_combine_backward(to_dev_bf16(dout), to_dev_bf16(y), to_dev(row_of), to_dev(row_token), to_dev(w), True,
                                              bf16=True)
    assert fp8bs.fp8bs_get_device_status() == 7
    assert fp8bs.fp8bs_get_device_status() == 0
    clean = row_of.copy()
    clean[2, 1] = -1
    want = _expected_dy(dout, clean, w, rows)
    want[5] = bf16_of(f32(dout[0]) * np.float32(5.0))
    assert np.array_equal(bits_of(dy), want)
    check_codes(q, s, want, True, "dy")
    _, ref, mag = train.combine_backward(f32(dout), f32(y), clean, w, rows)
    check_near(to_host(dw), ref, mag, _dot_steps(N), 0.0, "dw")


def test_combine_gradient_of_no_tokens_bf16_alone_and_strides():
    torch, fp8bs = require_gpu()
    rows, N = 128, 256
    none = torch.empty((0, N), dtype=torch.bfloat16, device="cuda:0")
    q, s, dy, dw = fp8bs.moe_combine_backward(none, torch.empty((rows, N), dtype=torch.bfloat16, device="cuda:0"),
                                              torch.empty((0, 2), dtype=torch.int32, device="cuda:0"),
                                              torch.full((rows,), -1, dtype=torch.int32, device="cuda:0"),
                                              torch.empty((0, 2), device="cuda:0"), bf16=True)
    assert not q.any() and not s.any() and not dy.any() and dw.shape == (0, 2)
    T, E, k, N = 20, 4, 2, 72
    row_token, row_of, rows = _layout(T, E, k, 9)
    wide = to_dev_bf16(synth.normal_bf16((T, N + 8), 1.0, 9, 4))
    w = np.random.default_rng(1).random((T, k)).astype(np.float32)
    dy = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda:0")
    fp8bs.fp8bs_moe_combine_backward(wide, T, N, N + 8, None, rows, to_dev(row_of), to_dev(row_token), to_dev(w), k, dy, None, None, 0,
                                     None)
    assert np.array_equal(bits_of(dy), _expected_dy(bits_of(wide[:, :N].contiguous()), row_of, w, rows))


@pytest.mark.parametrize("T", [9, 400])
def test_weights_far_from_one(T):
    """Weights and rows of any size whose product is a number: w / s alone may be none."""
    torch, fp8bs = require_gpu()
    E, k, N = 4, 3, 256
    row_token, row_of, rows = _layout(T, E, k, 11, 0.0)
    up = np.array([-125, -120, -60, 0, 60, 100])[np.arange(T) % 6]
    x = f32(synth.normal_bf16((T, N), 1.0, 13, 4)).astype(np.float64)
    dout = bf16_of((np.clip(x, -8, 8) * 2.0 ** up[:, None]).astype(np.float32))
    w = np.stack([2.0 ** (-up - 3 + 20.0 * j) for j in (-1, 0, 1)], 1)
    w = (np.clip(w, 2.0 ** -120, 2.0 ** 126) * 1.3).astype(np.float32)
    want = _expected_dy(dout, row_of, w, rows)
    assert np.isfinite(f32(want)).all() and (w[:, 0] > 2.0 ** 90).any()
    y = synth.normal_bf16((rows, N), 2.0 ** -20, 14, 1)
    for pow2 in (True, False):
        q, s, dy, _ = fp8bs.moe_combine_backward(to_dev_bf16(dout), to_dev_bf16(y), to_dev(row_of), to_dev(row_token), to_dev(w),
                                                 pow2, bf16=True)
        assert np.array_equal(bits_of(dy), want)
        check_codes(q, s, want, pow2, "dy")
    assert fp8bs.fp8bs_get_device_status() == 0


@pytest.mark.parametrize("T,E,k,N", [(1, 8, 2, 8), (3, 5, 1, 264), (37, 16, 4, 640), (300, 32, 8, 7168), (129, 64, 13, 128), (5, 64, 64, 1000)])
@pytest.mark.parametrize("add", [False, True])
def test_dispatch_gradient(T, E, k, N, add):
    torch, fp8bs = require_gpu()
    _, row_of, rows = _layout(T, E, k, T)
    row_of[0, 0] = rows + 3          # beyond the rows: adds nothing
    d, a = synth.normal_bf16((rows, N), 1e-3, 1, 4, outliers=True), synth.normal_bf16((T, N), 1e-3, 2, 4)
    ad = to_dev_bf16(a) if add else None
    dx = fp8bs.moe_dispatch_backward(to_dev_bf16(d), to_dev(row_of), ad)
    ref, mag = train.dispatch_backward(f32(d), row_of, f32(a) if add else None)
    check_near(to_host(dx), ref, mag, k + 1, BF16_HALF, "dx")
    if add:                          # over the addend itself
        fp8bs.fp8bs_moe_dispatch_backward(to_dev_bf16(d), rows, N, to_dev(row_of), T, k, ad, ad)
        assert torch.equal(ad, dx)
    else:                            # the combine with weights of one
        assert torch.equal(dx, _combine(torch, fp8bs, to_dev_bf16(d), to_dev(row_of)))


def _combine(torch, fp8bs, d, row_of):
    from fp8_fine_grained_fp8bs_gb300 import moe
    return moe._kernel_combine(d, row_of, torch.ones(row_of.shape, device="cuda:0"))


def test_graph():
    """Both gradients captured once, replayed on other inputs and another layout."""
    torch, fp8bs = require_gpu()
    T, E, k, N = 60, 8, 2, 256

    def inputs(seed):
        row_token, row_of, rows = _layout(T, E, k, seed)
        g = np.random.default_rng(seed)
        return [to_dev_bf16(synth.normal_bf16((T, N), 1.0, seed, 4)), to_dev_bf16(synth.normal_bf16((rows, N), 1.0, seed + 1, 1)),
                to_dev(row_of), to_dev(row_token), to_dev(g.random((T, k)).astype(np.float32))]

    def step(dout, y, row_of, row_token, w):
        q, s, _, dw = fp8bs.moe_combine_backward(dout, y, row_of, row_token, w, True)
        return q, s, dw, fp8bs.moe_dispatch_backward(y, row_of, dout)

    a, b = inputs(1), inputs(50)
    want = [t.clone() for t in step(*b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(*a)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, want))
