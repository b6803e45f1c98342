"""A training step of the MoE layer with 8-bit experts as it is used: norm with the residual, route, lay out, dispatch,
products, combine; then backward through all of it to the experts' weights, the router's logits, the gain and the
residual stream.

Each stage is checked against float64 on the stage before it as the GPU left it; the layer's functions must give the
bits of the stages called one by one.  The whole step is then compared with the same layer in float64 without any
quantisation."""
import numpy as np
import pytest

import oracle
from oracle import route, train
from fp8_fine_grained_fp8bs_gb300 import moe, synth
from _gpu import require_gpu, to_dev, to_dev_bf16, to_host
from _parity import check_bf16, check_f32
from _train import BF16_HALF, bits_of, check_codes, check_near, f32

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _inputs(T, E, H, I, seed=0):
    x, res = synth.normal_bf16((T, H), 1.0, seed, 1), synth.normal_bf16((T, H), 1.0, seed, 2)
    wg, wd = synth.normal_bf16((E, 2 * I, H), 0.06, seed, 5), synth.normal_bf16((E, H, I), 0.06, seed, 6)
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)).astype(np.float32)
    gain = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    dout = synth.normal_bf16((T, H), 1e-2, seed, 4)
    return x, res, wg, wd, z, gain, dout


def _values(q, s):
    """The numbers that codes [M, K] and kb-major scales [K/128, M] stand for."""
    return oracle.dequantize_1x128(to_host(q), to_host(s).T).astype(np.float64)


def _weight_values(q, s):
    return np.stack([oracle.e4m3_decode(a).astype(np.float64) * np.repeat(np.repeat(b, 128, 0), 128, 1).astype(np.float64)
                     for a, b in zip(to_host(q), to_host(s))])


@pytest.mark.parametrize("T,E,H,I,k", [(1, 4, 128, 128, 2), (70, 6, 384, 128, 3), (300, 12, 256, 256, 4)])
def test_step_stage_by_stage(T, E, H, I, k):
    torch, fp8bs = require_gpu()
    x, res, wg, wd, z, gain, dout = _inputs(T, E, H, I)
    experts = moe.quantize_experts_fp8(to_dev_bf16(wg), to_dev_bf16(wd))
    for plain, transposed in ((experts.gate_up, experts.gate_up_t), (experts.down, experts.down_t)):
        assert torch.equal(plain[0].transpose(1, 2), transposed[0]) and torch.equal(plain[1].transpose(1, 2), transposed[1])
    gd, add = to_dev(gain), to_dev_bf16(dout)
    q, s, _, r, rstd = fp8bs.rmsnorm_quantize(to_dev_bf16(x), gd, to_dev_bf16(res), EPS, pow2=True)
    out, saved = moe.moe_layer_fp8(q, s, to_dev(z), experts, k, scale=1.5, alpha=1e-2)
    one = torch.ones(1, device="cuda:0")
    dx, dz, dwg, dwd = moe.moe_layer_fp8_backward(add, saved, experts, one, None)
    dr, dgain = fp8bs.rmsnorm_backward(dx, r, gd, rstd, add)
    assert fp8bs.fp8bs_get_device_status() == 0

    # forward, stage by stage
    idx, w, counts, tokens, _ = saved.route
    off, tok, row = (to_host(t) for t in saved.layout)
    ri, rw, *_ = route.route(z, k, 0, scale=1.5)
    assert np.array_equal(to_host(idx), ri) and np.allclose(to_host(w), rw, rtol=1e-5, atol=0)
    for got, ref in zip((off, tok, row), route.layout(ri, E, len(tok))):
        assert np.array_equal(got, ref)
    xv, here = _values(*saved.x), tok >= 0
    assert np.array_equal(xv[here], _values(q, s)[tok[here]]) and not xv[~here].any()
    wgv, wdv = _weight_values(*experts.gate_up), _weight_values(*experts.down)
    h, y, vv = to_host(saved.h), to_host(saved.y), _values(*saved.v)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        check_bf16(h[lo:hi], xv[lo:hi] @ wgv[e].T, np.abs(xv[lo:hi]) @ np.abs(wgv[e]).T, f"gate/up of expert {e}")
        check_bf16(y[lo:hi], vv[lo:hi] @ wdv[e].T, np.abs(vv[lo:hi]) @ np.abs(wdv[e]).T, f"down of expert {e}")
    _, exact, mag = oracle.moe_combine(y, row, to_host(w))
    check_bf16(to_host(out), exact, mag, "combine")

    # backward, stage by stage
    dyq, sdy, dy, dw = fp8bs.moe_combine_backward(add, saved.y, saved.layout[2], saved.layout[1], w, True, bf16=True)
    _, dw_ref, dw_mag = train.combine_backward(f32(dout), y, row, to_host(w), len(tok))
    check_near(to_host(dw), dw_ref, dw_mag, 25, 0.0, "dw")
    check_codes(dyq, sdy, bits_of(dy), True, "dy")
    dv = fp8bs.grouped_gemm(dyq, sdy, saved.layout[0], *experts.down_t, pow2=True)
    dhq, sdh, _ = fp8bs.swiglu_backward_quantize(saved.h, dv, saved.layout[1], True)
    drows = fp8bs.grouped_gemm(dhq, sdh, saved.layout[0], *experts.gate_up_t, pow2=True)
    dyv, dhv = _values(dyq, sdy), _values(dhq, sdh)
    live = slice(0, off[E])
    dh_ref, dh_mag = train.swiglu_backward(h[live], np.where(here[live, None], to_host(dv)[live], 0.0), I)
    dh_ref[~here[live]] = 0.0
    assert np.linalg.norm(dhv[live] - dh_ref) <= 2.0 ** -4 * np.linalg.norm(dh_ref) + 1e-30   # E4M3's half step, relative
    a_dy, a_v, a_dh, a_x = ([*fp8bs.requant_1x128_to_128x1(*t)] for t in ((dyq, sdy), saved.v, (dhq, sdh), saved.x))
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        check_bf16(to_host(dv)[lo:hi], dyv[lo:hi] @ wdv[e], np.abs(dyv[lo:hi]) @ np.abs(wdv[e]), f"dv of expert {e}")
        check_bf16(to_host(drows)[lo:hi], dhv[lo:hi] @ wgv[e], np.abs(dhv[lo:hi]) @ np.abs(wgv[e]), f"rows of expert {e}")
    t = [_values(*p) for p in (a_dy, a_v, a_dh, a_x)]
    check_f32(to_host(dwd), *train.grouped_wgrad(t[0], t[1], off), "dw_down")
    check_f32(to_host(dwg), *train.grouped_wgrad(t[2], t[3], off), "dw_gate_up")
    ref, mag = train.dispatch_backward(to_host(drows), row)
    check_near(to_host(dx), ref, mag, k + 1, BF16_HALF, "dx")
    ref, mag, ref_g, mag_g = train.rmsnorm_backward(to_host(dx), to_host(r), gain, to_host(rstd), f32(dout))
    check_near(to_host(dr), ref, mag, 80, BF16_HALF, "dr")
    check_near(to_host(dgain), ref_g, mag_g, T / 304 + 60, 0.0, "dgain")
    assert torch.equal(dz, fp8bs.moe_route_backward(to_dev(z), idx, dw, scale=1.5, alpha=1e-2, counts=counts, tokens=tokens, dloss=one))


def _float64_layer(torch, x, res, wg, wd, z, gain, dout, idx, alpha):
    """The step in float64 without quantisation, by torch's autograd: the gradients of everything."""
    v = [torch.tensor(np.asarray(a, np.float64), requires_grad=True) for a in (f32(x), f32(res), f32(wg), f32(wd), z, gain)]
    xt, rt, wgt, wdt, zt, gt = v
    r = xt + rt
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * gt
    p = torch.softmax(zt, 1)
    w = p.gather(1, idx) / p.gather(1, idx).sum(1, keepdim=True)
    out = r.clone()
    I = wdt.shape[2]
    for e in range(wgt.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            h = n[t] @ wgt[e].t()
            y = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ wdt[e].t()
            out = out.index_add(0, t, y * w[t, j, None])
    T, E, k = idx.shape[0], wgt.shape[0], idx.shape[1]
    load = torch.bincount(idx.reshape(-1), minlength=E).double() * E / (k * T)
    loss = (out * torch.tensor(f32(dout).astype(np.float64))).sum() + alpha * (load * p.mean(0)).sum()
    return torch.autograd.grad(loss, v)


def test_step_against_float64_without_quantisation():
    """E4M3 keeps a value to 2^-4 relative.  A gradient here passes through at most five quantised operands one
    after the other, and twice as many meet in a sum's terms, independent of one another: in norm each product's
    error is below 2^-4 sqrt(2 * 5) = 0.2 of it; a wrong formula is off by as much as the gradient itself."""
    torch, fp8bs = require_gpu()
    T, E, H, I, k, alpha = 256, 8, 512, 256, 2, 0.3
    x, res, wg, wd, z, gain, dout = _inputs(T, E, H, I, 3)
    experts = moe.quantize_experts_fp8(to_dev_bf16(wg), to_dev_bf16(wd))
    gd, add = to_dev(gain), to_dev_bf16(dout)
    q, s, _, r, rstd = fp8bs.rmsnorm_quantize(to_dev_bf16(x), gd, to_dev_bf16(res), EPS, pow2=True)
    out, saved = moe.moe_layer_fp8(q, s, to_dev(z), experts, k, alpha=alpha)
    dx, dz, dwg, dwd = moe.moe_layer_fp8_backward(add, saved, experts, torch.ones(1, device="cuda:0"))
    dr, dgain = fp8bs.rmsnorm_backward(dx, r, gd, rstd, add)
    ref = _float64_layer(torch, x, res, wg, wd, z, gain, dout, saved.route[0].cpu().long(), alpha)
    assert torch.equal(ref[0], ref[1])
    for name, got, want in (("dr", dr, ref[0]), ("dw_gate_up", dwg, ref[2]), ("dw_down", dwd, ref[3]), ("dlogits", dz, ref[4]),
                            ("dgain", dgain, ref[5])):
        off = float((got.double().cpu() - want).norm() / want.norm())
        assert off < 0.2, (name, off)
    # added to gradients that are there, and the residual's gradient to dx
    twice = moe.moe_layer_fp8_backward(add, saved, experts, torch.ones(1, device="cuda:0"), add, dwg.clone(), dwd.clone())
    assert torch.allclose(twice[2], 2 * dwg, rtol=1e-6, atol=1e-12) and torch.allclose(twice[3], 2 * dwd, rtol=1e-6, atol=1e-12)
    assert torch.allclose(twice[0].float(), dx.float() + add.float(), rtol=2.0 ** -6, atol=1e-4)


def test_masked_tokens_and_serving_weights():
    """A masked token gets nothing and gives nothing back; weights quantised for serving run forward."""
    torch, fp8bs = require_gpu()
    T, E, H, I, k = 40, 6, 256, 128, 2
    x, res, wg, wd, z, gain, dout = _inputs(T, E, H, I, 5)
    valid = torch.ones(T, dtype=torch.uint8, device="cuda:0")
    valid[[0, 7]] = 0
    q, s, *_ = fp8bs.rmsnorm_quantize(to_dev_bf16(x), to_dev(gain), to_dev_bf16(res), EPS, pow2=True)
    experts = moe.quantize_experts_fp8(to_dev_bf16(wg), to_dev_bf16(wd))
    out, saved = moe.moe_layer_fp8(q, s, to_dev(z), experts, k, valid=valid)
    dx, dz, dwg, dwd = moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts)
    for t in (out, dx, dz):
        assert not t[[0, 7]].any() and t[1].any()
    serving = moe.quantize_experts_fp8(to_dev_bf16(wg), to_dev_bf16(wd), train=False)
    assert serving.gate_up_t is None and torch.equal(serving.down[0], experts.down[0]) and torch.equal(serving.down[1], experts.down[1])
    assert torch.equal(moe.moe_layer_fp8(q, s, to_dev(z), serving, k, valid=valid)[0], out)
    assert fp8bs.fp8bs_get_device_status() == 0


def test_step_in_a_graph():
    """The whole step captured once and replayed on other inputs, beside an eager step of the same tensors."""
    torch, fp8bs = require_gpu()
    T, E, H, I, k = 64, 4, 256, 128, 2
    a, b = _inputs(T, E, H, I, 6), _inputs(T, E, H, I, 7)
    experts = moe.quantize_experts_fp8(to_dev_bf16(a[2]), to_dev_bf16(a[3]))
    gain, one = to_dev(a[5]), torch.ones(1, device="cuda:0")
    held = [to_dev_bf16(a[0]), to_dev_bf16(a[1]), to_dev(a[4]), to_dev_bf16(a[6])]

    def step(x, res, z, dout):
        q, s, _, r, rstd = fp8bs.rmsnorm_quantize(x, gain, res, EPS, pow2=True)
        out, saved = moe.moe_layer_fp8(q, s, z, experts, k, alpha=0.1)
        dx, dz, dwg, dwd = moe.moe_layer_fp8_backward(dout, saved, experts, one)
        return (out, dz, dwg, dwd, *fp8bs.rmsnorm_backward(dx, r, gain, rstd, dout))

    eager = step(*held)
    kept = [t.clone() for t in eager]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(*held)
    torch.cuda.synchronize()
    for t, v in zip(held, (to_dev_bf16(b[0]), to_dev_bf16(b[1]), to_dev(b[4]), to_dev_bf16(b[6]))):
        t.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(eager, kept))
    assert all(torch.equal(p, q) for p, q in zip(out, step(*held)))
    assert fp8bs.fp8bs_get_device_status() == 0


def test_rows_behind_the_last_segment_do_not_matter():
    """The products leave the rows behind the last expert's as they were: memory full of NaN there changes no bit."""
    torch, fp8bs = require_gpu()
    T, E, H, I, k = 90, 6, 256, 128, 2
    x, res, wg, wd, z, gain, dout = _inputs(T, E, H, I, 8)
    z[:, 3:] -= 100.0                      # few experts are chosen: most of the rows are behind the last segment
    experts = moe.quantize_experts_fp8(to_dev_bf16(wg), to_dev_bf16(wd))
    held = [to_dev_bf16(x), to_dev(gain), to_dev_bf16(res), to_dev(z), to_dev_bf16(dout)]

    def step(fill):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        for n in (1 << 19, 1 << 20):       # what the allocator hands out again, small pieces and large
            del_me = [torch.full((n,), fill, dtype=torch.uint8, device="cuda:0") for _ in range(64)]
            del del_me
        xd, gd, rd, zd, add = held
        q, s, _, r, rstd = fp8bs.rmsnorm_quantize(xd, gd, rd, EPS, pow2=True)
        out, saved = moe.moe_layer_fp8(q, s, zd, experts, k)
        assert int(saved.layout[0][-1]) < len(saved.layout[1])
        return (out, *moe.moe_layer_fp8_backward(add, saved, experts))

    want = step(0)
    got = step(0xFF)
    assert fp8bs.fp8bs_get_device_status() == 0
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and all(bool(torch.isfinite(t.float()).all()) for t in got)


def test_backward_refusals():
    """Refused before anything is launched or added to."""
    torch, fp8bs = require_gpu()
    T, E, H, I, k = 20, 4, 256, 128, 2
    x, res, wg, wd, z, gain, dout = _inputs(T, E, H, I, 9)
    experts = moe.quantize_experts_fp8(to_dev_bf16(wg), to_dev_bf16(wd))
    q, s, *_ = fp8bs.rmsnorm_quantize(to_dev_bf16(x), to_dev(gain), to_dev_bf16(res), EPS, pow2=True)
    _, saved = moe.moe_layer_fp8(q, s, to_dev(z), experts, k)
    down = torch.zeros((E, H, I), device="cuda:0")
    up = torch.zeros((E, 2 * I, H), device="cuda:0")
    for bad in (up.bfloat16(), up[:, :I], up.transpose(1, 2)):
        with pytest.raises(ValueError, match="dw_gate_up"):
            moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts, dw_gate_up=bad, dw_down=down)
    with pytest.raises(ValueError, match="dw_down"):
        moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts, dw_gate_up=up, dw_down=down[:2])
    with pytest.raises(ValueError, match="dloss"):
        moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts, torch.ones(1, device="cuda:0"))
    with pytest.raises(ValueError, match="serving"):
        moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts._replace(gate_up_t=None))
    torch.cuda.synchronize()
    assert not down.any() and not up.any()
