"""The allocating functions refuse tensors whose type, shape or strides the C
entry points could not see."""
import pytest

from _gpu import require_gpu

pytestmark = pytest.mark.gpu


def test_refusals():
    torch, fp8bs = require_gpu()
    dev = "cuda:0"
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    a, b = fp8bs.quantize_fp4(x), fp8bs.quantize_fp4(torch.zeros((8, 64), dtype=torch.bfloat16, device=dev))
    z = torch.zeros((4, 16), device=dev)
    idx, w = fp8bs.moe_route(z, 2)
    for call in (
            lambda: fp8bs.quantize_fp4(x.float()), lambda: fp8bs.quantize_fp4(x.cpu()), lambda: fp8bs.quantize_fp4(x.t()),
            lambda: fp8bs.quantize_fp4(x, rows=torch.zeros(3, dtype=torch.int64, device=dev)),
            lambda: fp8bs.swiglu_quantize_fp4(torch.zeros((4, 128), dtype=torch.bfloat16, device=dev),
                                              live=torch.zeros(3, dtype=torch.int32, device=dev)),
            lambda: fp8bs.dequantize_fp4(a[0], a[1][:512], a[2][:3]),
            lambda: fp8bs.gemm_fp4(a, (b[0][:, :16], b[1], b[2])), lambda: fp8bs.gemm_fp4(a, b, fp8bs.FP4_UE8M0X32, out=z),
            lambda: fp8bs.gemm_fp4(a, b, out=torch.zeros((4, 9), device=dev)),
            lambda: fp8bs.gemm_fp4((a[0], a[1], None), b),
            lambda: fp8bs.grouped_gemm_fp4(a, torch.zeros(3, dtype=torch.int32, device=dev), tuple(t[None] for t in b)),
            lambda: fp8bs.moe_route(z.half(), 2), lambda: fp8bs.moe_route(z, 2, valid=torch.ones(5, dtype=torch.uint8, device=dev)),
            lambda: fp8bs.moe_route(z, 2, 1, bias=torch.zeros(4, device=dev)),
            lambda: fp8bs.moe_route_backward(z, idx, w.double()), lambda: fp8bs.moe_route_backward(z, idx[:3], w),
            lambda: fp8bs.moe_layout(idx.long(), 16)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fp8bs.moe_route(z, 17), lambda: fp8bs.moe_layout(idx, 0), lambda: fp8bs.moe_route(z, 2, 0, bias=z[0]),
                 lambda: fp8bs.fp4_scale_bytes(4, 65, 0)):
        with pytest.raises(fp8bs.Fp8bsError):
            call()


def test_scratch_on_another_stream():
    """A call queued on another stream keeps its scratch memory until it has run."""
    torch, fp8bs = require_gpu()
    z = torch.randn((20000, 64), device="cuda:0")
    ref = fp8bs.moe_route(z, 4, alpha=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = fp8bs.moe_route(z, 4, alpha=0.1, stream=side)
        torch.empty(1 << 22, dtype=torch.uint8, device="cuda:0").fill_(0xFF)    # would take freed scratch at once
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    offsets, row_token, row_of = fp8bs.moe_layout(ref[0], 64)
    got = fp8bs.moe_layout(ref[0], 64, stream=side.cuda_stream)
    torch.empty(1 << 20, dtype=torch.uint8, device="cuda:0").fill_(0xFF)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((offsets, row_token, row_of), got))
