"""The MoE layer with 4-bit experts as it is used: route, lay out, gather and
quantise, grouped GEMM, SwiGLU and quantise, grouped GEMM, combine.

Each stage is checked against the oracle on the stage before it as the GPU
left it (codes bit for bit, products within the GEMM tolerances of
tests/_parity.py, the combine within one BF16 ulp); the layer's function must
then give the bits of the stages called one by one."""
import numpy as np
import pytest

import oracle
from oracle import fp4, route
from fp8_fine_grained_fp8bs_gb300 import moe, synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _parity import assert_bytes_equal, check_bf16

pytestmark = pytest.mark.gpu


def _inputs(T, E, H, I, seed=0):
    x = synth.normal_bf16((T, H), 1.0, seed, 1, outliers=True)
    wg = synth.normal_bf16((E, 2 * I, H), 0.05, seed, 5)
    wd = synth.normal_bf16((E, H, I), 0.05, seed, 6)
    z = np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32)
    return x, wg, wd, z


def _values(bits, fmt):
    return fp4.values(*fp4.quantize(oracle.bf16_bits_to_f32(bits).astype(np.float32), fmt), fmt)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 256, 128, 2), (70, 6, 320, 192, 3), (300, 12, 192, 64, 4)])
def test_layer_stage_by_stage(T, E, H, I, k, fmt):
    torch, fp8bs = require_gpu()
    x, wg, wd, z = _inputs(T, E, H, I)
    experts = moe.quantize_experts_fp4(to_dev_bf16(wg), to_dev_bf16(wd), fmt)
    out, (idx, w) = moe.moe_layer_fp4(to_dev_bf16(x), to_dev(z), experts, k, fmt, scale=1.5)

    ri, rw, *_ = route.route(z, k, 0, scale=1.5)
    assert np.array_equal(to_host(idx), ri) and np.allclose(to_host(w), rw, rtol=1e-5, atol=0)
    offsets, row_token, row_of = fp8bs.moe_layout(idx, E)
    off, tok, row = (to_host(t) for t in (offsets, row_token, row_of))
    for got, ref in zip((off, tok, row), route.layout(ri, E, len(tok))):
        assert np.array_equal(got, ref)

    a = fp8bs.quantize_fp4(to_dev_bf16(x), fmt, rows=row_token)
    xr = np.where((tok >= 0)[:, None], oracle.bf16_bits_to_f32(x)[np.maximum(tok, 0)], np.float32(0)).astype(np.float32)
    assert_bytes_equal(to_host(a[0]), fp4.pack(fp4.quantize(xr, fmt)[0]), "gathered rows")
    h = fp8bs.grouped_gemm_fp4(a, offsets, experts[0], fmt)
    q = fp8bs.swiglu_quantize_fp4(h, fmt, live=row_token)
    y = fp8bs.grouped_gemm_fp4(q, offsets, experts[1], fmt)
    assert fp8bs.fp8bs_get_device_status() == 0
    gate, up = h[:, :I].float(), h[:, I:].float()
    v = to_host(((gate / (1.0 + torch.exp(-gate))) * up).to(torch.bfloat16).float())    # no gate below -64 here
    va = fp4.values(*fp4.quantize(xr, fmt), fmt)
    vr = np.where((tok >= 0)[:, None], v, np.float32(0)).astype(np.float32)
    assert_bytes_equal(to_host(q[0]), fp4.pack(fp4.quantize(vr, fmt)[0]), "swiglu rows")
    vq = fp4.values(*fp4.quantize(vr, fmt), fmt)
    hh, yy = to_host(h), to_host(y)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        check_bf16(hh[lo:hi], *fp4.gemm(va[lo:hi], _values(wg[e], fmt)), f"gate/up of expert {e}")
        check_bf16(yy[lo:hi], *fp4.gemm(vq[lo:hi], _values(wd[e], fmt)), f"down of expert {e}")
    ref, exact, mag = oracle.moe_combine(yy, row, to_host(w))
    check_bf16(to_host(out), exact, mag, "combine")
    whole = moe._kernel_combine(y, row_of, w)
    assert torch.equal(out, whole)


def test_layer_in_a_graph_and_masked_tokens():
    """Captured once, replayed on other inputs; a masked token's output is zero."""
    torch, fp8bs = require_gpu()
    T, E, H, I, k = 40, 8, 256, 128, 2
    x, wg, wd, z = _inputs(T, E, H, I, 1)
    x2, _, _, z2 = _inputs(T, E, H, I, 2)
    experts = moe.quantize_experts_fp4(to_dev_bf16(wg), to_dev_bf16(wd))
    xd, zd = to_dev_bf16(x), to_dev(z)
    valid = torch.ones(T, dtype=torch.uint8, device="cuda:0")
    valid[3] = 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_layer_fp4(xd, zd, experts, k, valid=valid)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, (idx, w) = moe.moe_layer_fp4(xd, zd, experts, k, valid=valid)
    torch.cuda.synchronize()
    xd.copy_(to_dev_bf16(x2))
    zd.copy_(to_dev(z2))
    graph.replay()
    torch.cuda.synchronize()
    ref, (ri, rw) = moe.moe_layer_fp4(to_dev_bf16(x2), to_dev(z2), experts, k, valid=valid)
    assert torch.equal(out, ref) and torch.equal(idx, ri) and torch.equal(w, rw)
    assert not out[3].any() and torch.all(idx[3] == -1)


def test_router_gradient_through_the_layer_against_differences():
    """The training use: the loss L = <out, r> + balance loss, with the experts'
    outputs held fixed as the combine's gradient holds them.  Central
    differences of the float32 kernels, step h: the weights' rounding of 2^-23
    |y r| summed over H terms and divided by 2h, plus h^2 / 6 of a third
    derivative below 8 |y r| (k <= 3, softmax), stay under 2e-3 of the scale."""
    torch, fp8bs = require_gpu()
    T, E, H, k, h = 12, 10, 64, 3, 1e-2
    rng = np.random.default_rng(3)
    z = rng.standard_normal((T, E)).astype(np.float32)
    y = torch.from_numpy(rng.standard_normal((T, k, H)).astype(np.float32)).to("cuda:0")     # expert outputs, by slot
    r = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to("cuda:0")
    kw = dict(score=0, scale=1.3, alpha=0.5)
    idx, w, counts, tokens, loss = fp8bs.moe_route(to_dev(z), k, **kw)
    dw = torch.einsum("tkh,th->tk", y, r).contiguous()
    one = torch.ones(1, device="cuda:0")
    dz = to_host(fp8bs.moe_route_backward(to_dev(z), idx, dw, counts=counts, tokens=tokens, dloss=one, **kw))

    def value(zz):
        i2, w2, _, _, l2 = fp8bs.moe_route(to_dev(zz.astype(np.float32)), k, **kw)
        same = torch.equal(i2, idx)
        return float((w2.double() * dw.double()).sum() + l2.double()), same

    scale, checked = float(dw.abs().max()), 0
    for t in range(T):
        for e in range(E):
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            (a, sa), (b, sb) = value(up), value(down)
            if sa and sb:                       # the choice must not change within the step
                step = float(up[t, e]) - float(down[t, e])
                assert abs((a - b) / step - dz[t, e]) < 2e-3 * scale
                checked += 1
    assert checked > T * E // 2
