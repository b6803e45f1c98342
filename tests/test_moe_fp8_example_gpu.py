"""The training example: it runs, and its gradients are those of the block in float64."""
import importlib.util
import os
import subprocess
import sys

import pytest

from _gpu import require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "moe_fp8_train.py")


def test_example_runs():
    require_gpu()
    out = subprocess.run([sys.executable, PATH, "--tokens", "300", "--experts", "6", "--hidden", "256", "--inner", "128", "--top-k", "2",
                          "--steps", "2"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("step ") == 2


def test_example_gradients():
    """Against float64's autograd on unquantised weights, with the experts as the block chose them.  A gradient
    passes through at most five 8-bit operands, each within 2^-4 of its value and as many again in a sum's other
    factor: 2^-4 sqrt(2 * 5) = 0.2 of the gradient's norm, as in test_moe_fp8_train_gpu."""
    torch, fp8bs = require_gpu()
    spec = importlib.util.spec_from_file_location("moe_fp8_train", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    torch.manual_seed(1)
    T, E, H, I, k = 320, 8, 512, 256, 2
    params, x, residual = ex.make(T, E, H, I)
    params["gain"] += 0.2 * torch.randn(H, device=x.device)
    experts = ex.quantise(params)
    out, kept = ex.forward(params, experts, x, residual, k)
    dout = (torch.randn(T, H, device=x.device) / T).bfloat16()
    dr, grads = ex.backward(params, experts, dout, kept)
    assert fp8bs.fp8bs_get_device_status() == 0

    idx = kept[3].route[0].long()
    v = {n: p.double().requires_grad_() for n, p in params.items()}
    r = (x + residual).double().requires_grad_()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + ex.EPS) * v["gain"]
    p = torch.softmax(y @ v["router"].t(), 1)
    w = p.gather(1, idx) / p.gather(1, idx).sum(1, keepdim=True)
    ref = r.clone()
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            gate, up = (y[t] @ v["gate_up"][e].t()).chunk(2, dim=1)
            ref = ref.index_add(0, t, ((torch.nn.functional.silu(gate) * up) @ v["down"][e].t()) * w[t, j, None])
    load = torch.bincount(idx.reshape(-1), minlength=E).double() * E / (k * T)
    loss = (ref * dout.double()).sum() + ex.ALPHA * (load * p.mean(0)).sum()
    want = torch.autograd.grad(loss, [r, *v.values()])
    assert float((out.double() - ref.detach()).norm() / ref.detach().norm()) < 0.2
    for name, got, ref in zip(["dr", *v], [dr, *grads.values()], want):
        off = float((got.double() - ref).norm() / ref.norm())
        assert off < 0.2, (name, off)
    # added up over two micro-batches
    twice = ex.backward(params, experts, dout, kept, {"gate_up": grads["gate_up"].clone(), "down": grads["down"].clone()})[1]
    assert torch.allclose(twice["gate_up"], 2 * grads["gate_up"], rtol=1e-6, atol=1e-12)
