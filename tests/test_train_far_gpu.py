"""The training step's operators where offsets pass 32 bits: the last rows of matrices of more than 2^32 elements give
the bits that the same rows give alone."""
import pytest

from fp8_fine_grained_fp8bs_gb300 import moe
from _gpu import require_gpu

pytestmark = pytest.mark.gpu
LAST = 200


def _far(torch, M, K, scale=1.0):
    """(all [M, K] bfloat16, zeros up to the last rows; those)."""
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda:0")
    x[-LAST:] = torch.randn((LAST, K), device="cuda:0") * scale
    return x, x[-LAST:].clone()


def _room(torch, gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB")


def test_norm_and_gradient():
    torch, fp8bs = require_gpu()
    _room(torch, 80)
    M, K = 270000, 16000                       # 4.3e9 elements
    torch.manual_seed(0)
    x, xs = _far(torch, M, K)
    res, rs = _far(torch, M, K)
    gain = torch.randn(K, device="cuda:0")
    q, s, y, r, rstd = fp8bs.rmsnorm_quantize(x, gain, res, pow2=True, bf16=True)
    want = fp8bs.rmsnorm_quantize(xs, gain, rs, pow2=True, bf16=True)
    for got, ref in zip((q[-LAST:], s[:, -LAST:], y[-LAST:], r[-LAST:], rstd[-LAST:]), want):
        assert torch.equal(got, ref)
    assert not q[:100].any() and not q[M // 2:M // 2 + 100].any()
    del q, s, x, res
    dx, dgain = fp8bs.rmsnorm_backward(y, r, gain, rstd, r)
    ref, dgain_ref = fp8bs.rmsnorm_backward(want[2], want[3], gain, want[4], want[3])
    assert torch.equal(dx[-LAST:], ref) and not dx[:M - LAST].any()
    # the same terms, summed in another order: LAST roundings of them at most
    bound = LAST * 2.0 ** -23 * (want[2].float() * want[3].float() * want[4][:, None]).abs().sum(0)
    assert bool(((dgain - dgain_ref).abs() <= bound).all())
    assert fp8bs.fp8bs_get_device_status() == 0


def test_swiglu_gradient():
    torch, fp8bs = require_gpu()
    _room(torch, 50)
    M, I = 540000, 4096                        # 4.4e9 elements of h
    torch.manual_seed(1)
    h, hs = _far(torch, M, 2 * I)
    dv, ds = _far(torch, M, I, 1e-3)
    q, s, dh = fp8bs.swiglu_backward_quantize(h, dv, pow2=True, bf16=True)
    for got, ref in zip((q[-LAST:], s[:, -LAST:], dh[-LAST:]), fp8bs.swiglu_backward_quantize(hs, ds, pow2=True, bf16=True)):
        assert torch.equal(got, ref)
    assert fp8bs.fp8bs_get_device_status() == 0


def test_gradients_of_combine_and_dispatch():
    torch, fp8bs = require_gpu()
    _room(torch, 50)
    T, k, N, rows = LAST // 2, 2, 8192, 540160     # 4.4e9 elements of y
    torch.manual_seed(2)
    y, ys = _far(torch, rows, N)
    dout = torch.randn((T, N), device="cuda:0").bfloat16()
    w = torch.rand((T, k), device="cuda:0")
    near = torch.randperm(LAST, device="cuda:0").int().view(T, k)
    token = torch.empty(LAST, dtype=torch.int32, device="cuda:0")
    token[near.long().reshape(-1)] = torch.arange(T, dtype=torch.int32, device="cuda:0").repeat_interleave(k)
    far_token = torch.full((rows,), -1, dtype=torch.int32, device="cuda:0")
    far_token[-LAST:] = token
    q, s, dy, dw = fp8bs.moe_combine_backward(dout, y, near + (rows - LAST), far_token, w, True, bf16=True)
    q2, s2, dy2, dw2 = fp8bs.moe_combine_backward(dout, ys, near, token, w, True, bf16=True)
    assert torch.equal(q[-LAST:], q2) and torch.equal(s[:, -LAST:], s2) and torch.equal(dy[-LAST:], dy2) and torch.equal(dw, dw2)
    assert not dy[:rows - LAST].any() and not q[:rows - LAST].any()
    assert torch.equal(fp8bs.moe_dispatch_backward(dy, near + (rows - LAST), dout), fp8bs.moe_dispatch_backward(dy2, near, dout))
    assert fp8bs.fp8bs_get_device_status() == 0


def test_weight_gradients():
    torch, fp8bs = require_gpu()
    _room(torch, 20)
    N, K, R, live = 1024, 256, (1 << 22) + 512, 256        # 4.3e9 codes of A
    torch.manual_seed(3)
    a, sa = torch.zeros((N, R), dtype=torch.uint8, device="cuda:0"), torch.zeros((R // 128, N), device="cuda:0")
    b, sb = torch.zeros((K, R), dtype=torch.uint8, device="cuda:0"), torch.zeros((R // 128, K), device="cuda:0")
    near = []
    for codes, scales, width in ((a, sa, N), (b, sb, K)):
        _, _, c, t = fp8bs.quantize_act(torch.randn((live, width), device="cuda:0").bfloat16(), True, True)
        codes[:, -live:], scales[-live // 128:] = c, t
        near += [c, t]
    off = torch.tensor([0, 128, R - live, R], dtype=torch.int32, device="cuda:0")
    d = fp8bs.grouped_wgrad(a, sa, b, sb, off)
    ref = fp8bs.grouped_wgrad(*near, torch.tensor([0, live], dtype=torch.int32, device="cuda:0"))
    assert torch.equal(d[2], ref[0]) and not d[:2].any() and bool(ref.any())
    assert fp8bs.fp8bs_get_device_status() == 0


def test_layer_of_no_tokens_and_of_one_expert():
    """The ends of the layer's ranges: nothing routed gives zeros, one expert is the dense product."""
    torch, fp8bs = require_gpu()
    H, I = 256, 128
    torch.manual_seed(4)
    for T, E, k in ((0, 4, 2), (1, 1, 1), (130, 1, 1), (3, 8, 8)):
        w1, w2 = (torch.randn(s, device="cuda:0").bfloat16() * 0.06 for s in ((E, 2 * I, H), (E, H, I)))
        experts = moe.quantize_experts_fp8(w1, w2)
        x = torch.randn((T, H), device="cuda:0").bfloat16()
        q, s, _, r, rstd = fp8bs.rmsnorm_quantize(x, torch.ones(H, device="cuda:0"), x, pow2=True)
        out, saved = moe.moe_layer_fp8(q, s, torch.randn((T, E), device="cuda:0"), experts, k)
        dx, dz, dwg, dwd = moe.moe_layer_fp8_backward(x, saved, experts)
        assert out.shape == dx.shape == (T, H) and dz.shape == (T, E) and dwg.shape == w1.shape and dwd.shape == w2.shape
        assert all(bool(torch.isfinite(t.float()).all()) for t in (out, dx, dz, dwg, dwd))
        if T == 0:
            assert not dwg.any() and not dwd.any()
        else:
            assert out.any() and dx.any() and dwg.any() and dwd.any()
        if k == E:                             # nothing is chosen: weights of equal sum, logits that may all move together
            assert bool((dz.float().sum(1).abs() <= 1e-5 * (1 + dz.float().abs().sum(1))).all())
        dr, dg = fp8bs.rmsnorm_backward(dx, r, torch.ones(H, device="cuda:0"), rstd)
        assert dr.shape == (T, H) and (T > 0 or not dg.any())
    assert fp8bs.fp8bs_get_device_status() == 0
