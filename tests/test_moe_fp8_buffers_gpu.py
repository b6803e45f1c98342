"""Gradient buffers that moe_layer_fp8_backward cannot add to are refused before it adds to the other one."""
import pytest

from fp8_fine_grained_fp8bs_gb300 import moe
from _gpu import require_gpu, to_dev, to_dev_bf16
from test_moe_fp8_train_gpu import _inputs

pytestmark = pytest.mark.gpu


def test_buffers_on_another_device():
    torch, fp8bs = require_gpu()
    T, E, H, I, k = 20, 4, 256, 128, 2
    x, res, wg, wd, z, gain, dout = _inputs(T, E, H, I, 9)
    experts = moe.quantize_experts_fp8(to_dev_bf16(wg), to_dev_bf16(wd))
    q, s, *_ = fp8bs.rmsnorm_quantize(to_dev_bf16(x), to_dev(gain), to_dev_bf16(res), 1e-6, pow2=True)
    _, saved = moe.moe_layer_fp8(q, s, to_dev(z), experts, k)
    down, up = torch.zeros((E, H, I), device="cuda:0"), torch.zeros((E, 2 * I, H), device="cuda:0")
    with pytest.raises(ValueError, match="dw_gate_up"):
        moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts, dw_gate_up=up.cpu(), dw_down=down)
    with pytest.raises(ValueError, match="dw_down"):
        moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts, dw_gate_up=up, dw_down=down.cpu())
    torch.cuda.synchronize()
    assert not down.any() and not up.any()
    _, _, up2, down2 = moe.moe_layer_fp8_backward(to_dev_bf16(dout), saved, experts, dw_gate_up=up, dw_down=down)
    assert up2 is up and down2 is down and up.any() and down.any()
    assert fp8bs.fp8bs_get_device_status() == 0
