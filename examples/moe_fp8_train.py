"""Training steps of a pre-norm mixture-of-experts block with 8-bit experts, as
a program writes them.

    python examples/moe_fp8_train.py [--tokens 2048] [--experts 16] [--hidden 2048] [--inner 1024] [--top-k 4] [--steps 5]

out = r + experts(norm(r)), r = x + residual: the norm adds the residual and
quantises for the experts in one pass, the router reads the norm's BF16 output,
every product of the experts runs in 8 bits, forward and backward.  The master
weights are float32; the experts are quantised once a step.  Prints the loss of
each step (a regression on random targets) and a step's time by its parts.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_fp8bs_gb300 as fp8bs  # noqa: E402
from fp8_fine_grained_fp8bs_gb300 import moe  # noqa: E402

EPS, ALPHA = 1e-6, 1e-2


def quantise(params):
    return moe.quantize_experts_fp8(params["gate_up"].bfloat16(), params["down"].bfloat16())


def forward(params, experts, x, residual, k):
    """(out [T, H] bfloat16, what backward needs)."""
    q, s, y, r, rstd = fp8bs.rmsnorm_quantize(x, params["gain"], residual, EPS, pow2=True, bf16=True)
    logits = y.float() @ params["router"].t()
    delta, saved = moe.moe_layer_fp8(q, s, logits, experts, k, alpha=ALPHA)
    return r + delta, (y, r, rstd, saved)


def backward(params, experts, dout, kept, grads=None):
    """Gradients of <out, dout> + the balance loss: of x (and the residual), and of each parameter; those of the
    experts are added to ``grads``, where given."""
    y, r, rstd, saved = kept
    one = torch.ones(1, device=dout.device)
    grads = grads or {}
    # the router's logits first: their gradient reaches the norm's output beside the experts'
    dx, dlogits, d_gate_up, d_down = moe.moe_layer_fp8_backward(dout, saved, experts, one, None, grads.get("gate_up"),
                                                                grads.get("down"))
    d_router = dlogits.t() @ y.float()
    dy = (dx.float() + dlogits @ params["router"]).bfloat16()
    dr, d_gain = fp8bs.rmsnorm_backward(dy, r, params["gain"], rstd, dres=dout)
    return dr, {"gain": d_gain, "router": d_router, "gate_up": d_gate_up, "down": d_down}


def make(T, E, H, I, dev="cuda:0"):
    params = {"gain": torch.ones(H, device=dev), "router": torch.randn(E, H, device=dev) / H ** 0.5,
              "gate_up": torch.randn(E, 2 * I, H, device=dev) / H ** 0.5, "down": torch.randn(E, H, I, device=dev) / I ** 0.5}
    x, residual = (torch.randn(T, H, device=dev).bfloat16() for _ in range(2))
    return params, x, residual


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 2048), ("experts", 16), ("hidden", 2048), ("inner", 1024), ("top-k", 4), ("steps", 5)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args()
    fp8bs.build()
    torch.manual_seed(0)
    params, x, residual = make(a.tokens, a.experts, a.hidden, a.inner)
    target = (x + residual).float() + torch.randn(a.tokens, a.hidden, device=x.device)
    rate = 0.02
    for step in range(a.steps):
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
        marks[0].record()
        experts = quantise(params)
        marks[1].record()
        out, kept = forward(params, experts, x, residual, a.top_k)
        marks[2].record()
        error = out.float() - target
        _, grads = backward(params, experts, (error / a.tokens).bfloat16(), kept)
        marks[3].record()
        for name, p in params.items():
            p -= rate * grads[name]
        torch.cuda.synchronize()
        parts = [marks[i].elapsed_time(marks[i + 1]) * 1e3 for i in range(3)]
        print(f"step {step}: loss {float(error.square().sum()) / (2 * a.tokens):.3f}, balance loss {float(kept[3].route[4]):.5f}, "
              f"quantise {parts[0]:.0f} us, forward {parts[1]:.0f} us, backward {parts[2]:.0f} us")
    status = fp8bs.fp8bs_get_device_status()
    if status:
        raise RuntimeError(f"device status {status}")


if __name__ == "__main__":
    main()
