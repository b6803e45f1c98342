"""A mixture-of-experts layer with 4-bit experts, forward and the router's
backward, as a program uses it.

    python examples/moe_fp4_layer.py [--tokens 256] [--experts 32] [--hidden 2048] [--inner 1024] [--top-k 8]

Quantises the experts once, runs the layer on a batch and on a single token
(captured in a CUDA graph, as decoding would), prints their times and the error
against the same layer in float32 with the BF16 weights, then one step of a
router's training: the gradient of <output, r> + balance loss with respect to
the router's weight.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_fp8bs_gb300 as fp8bs  # noqa: E402
from fp8_fine_grained_fp8bs_gb300 import moe  # noqa: E402


def reference(x, logits, w_gate_up, w_down, idx, w):
    """The layer in float32 on the BF16 weights, with the experts as chosen."""
    out = torch.zeros_like(x, dtype=torch.float32)
    for e in range(w_gate_up.shape[0]):
        token, slot = (idx == e).nonzero(as_tuple=True)
        if len(token):
            gate, up = (x[token].float() @ w_gate_up[e].float().t()).chunk(2, dim=1)
            y = (torch.nn.functional.silu(gate) * up) @ w_down[e].float().t()
            out.index_add_(0, token, y * w[token, slot, None])
    return out


def time_us(call, n=20):
    for _ in range(3):
        call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        call()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e3 / n


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 256), ("experts", 32), ("hidden", 2048), ("inner", 1024), ("top-k", 8)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args()
    fp8bs.build()
    torch.manual_seed(0)
    T, E, H, I, k = a.tokens, a.experts, a.hidden, a.inner, a.top_k
    dev = "cuda:0"
    x = torch.randn(T, H, device=dev).bfloat16()
    w_router = torch.randn(E, H, device=dev) / H ** 0.5
    w_gate_up = (torch.randn(E, 2 * I, H, device=dev) / H ** 0.5).bfloat16()
    w_down = (torch.randn(E, H, I, device=dev) / I ** 0.5).bfloat16()
    logits = x.float() @ w_router.t()

    for fmt, name in ((fp8bs.FP4_E4M3X16, "E4M3 scales per 16"), (fp8bs.FP4_UE8M0X32, "UE8M0 scales per 32")):
        experts = moe.quantize_experts_fp4(w_gate_up, w_down, fmt)
        out, (idx, w) = moe.moe_layer_fp4(x, logits, experts, k, fmt)
        ref = reference(x, logits, w_gate_up, w_down, idx, w)
        err = float((out.float() - ref).norm() / ref.norm())
        batch = time_us(lambda: moe.moe_layer_fp4(x, logits, experts, k, fmt))
        x1, z1 = x[:1].clone(), logits[:1].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            moe.moe_layer_fp4(x1, z1, experts, k, fmt)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                moe.moe_layer_fp4(x1, z1, experts, k, fmt)
        torch.cuda.current_stream().wait_stream(side)
        print(f"{name}: {T} tokens {batch:.1f} us, one token {time_us(graph.replay):.1f} us, "
              f"relative error against float32 {err:.3f}")

    # one step of the router's training, two packed sequences
    seq = torch.tensor([0, T // 3, T], dtype=torch.int32, device=dev)
    r = torch.randn(T, H, device=dev)
    experts = moe.quantize_experts_fp4(w_gate_up, w_down)
    out, (idx, w, counts, tokens, loss) = moe.moe_layer_fp4(x, logits, experts, k, seq=seq, alpha=1e-2)
    # d <out, r> / d w[t, j] = <expert output, r>: the layer with one slot's weight at a time
    dw = torch.stack([(reference(x, logits, w_gate_up, w_down, idx[:, j:j + 1], torch.ones_like(w[:, j:j + 1])) * r).sum(1)
                      for j in range(k)], dim=1).contiguous()
    dlogits = fp8bs.moe_route_backward(logits, idx, dw, seq=seq, alpha=1e-2, counts=counts, tokens=tokens,
                                       dloss=torch.ones(1, device=dev))
    dw_router = dlogits.t() @ x.float()
    busiest = int(counts.sum(0).max())
    print(f"balance loss {float(loss):.5f}, busiest expert {busiest} of {T * k} choices, "
          f"router gradient norm {float(dw_router.norm()):.4f}")
    status = fp8bs.fp8bs_get_device_status()
    if status:
        raise RuntimeError(f"device status {status}")


if __name__ == "__main__":
    main()
