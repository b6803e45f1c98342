"""Matrices without columns: what the calls return is not memory that nothing wrote."""
import pytest

from _gpu import require_gpu

pytestmark = pytest.mark.gpu


def _dirty(torch, n):
    """Memory full of ones' bits for the allocator to hand out again."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda:0") for _ in range(16)]
    del held


@pytest.mark.parametrize("slices", [False, True])
def test_combine_gradient_without_columns(slices):
    """The gate weights' gradient is a sum over no columns: zeros."""
    torch, fp8bs = require_gpu()
    T, k, rows = 37, 3, 128
    row_of = torch.arange(T * k, dtype=torch.int32, device="cuda:0").view(T, k)
    row_token = torch.full((rows,), -1, dtype=torch.int32, device="cuda:0")
    row_token[:T * k] = torch.arange(T * k, device="cuda:0").div(k, rounding_mode="floor").int()
    wide = 8 if slices else 0      # a slice of no columns has an address, an empty tensor has none
    args = (torch.empty((T, wide), dtype=torch.bfloat16, device="cuda:0")[:, :0],
            torch.empty((rows, wide), dtype=torch.bfloat16, device="cuda:0")[:, :0], row_of, row_token, torch.ones((T, k), device="cuda:0"))
    _dirty(torch, 4 * T * k)
    q, s, _, dw = fp8bs.moe_combine_backward(*args)
    assert q.shape == (rows, 0) and s.shape == (0, rows) and dw.shape == (T, k) and not dw.any()
    assert fp8bs.fp8bs_get_device_status() == 0


def test_norm_without_columns():
    """The rows' statistic is that of a mean of zero."""
    torch, fp8bs = require_gpu()
    M = 37
    x, gain = torch.empty((M, 8), dtype=torch.bfloat16, device="cuda:0")[:, :0], torch.empty(0, device="cuda:0")
    _dirty(torch, 4 * M)
    q, s, y, r, rstd = fp8bs.rmsnorm_quantize(x, gain, eps=0.25, bf16=True)
    assert q.shape == y.shape == r.shape == (M, 0) and s.shape == (0, M) and bool((rstd == 2.0).all())
    dx, dgain = fp8bs.rmsnorm_backward(x, r, gain, rstd)
    assert dx.shape == (M, 0) and dgain.shape == (0,)
