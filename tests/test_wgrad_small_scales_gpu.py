"""Re-tiling from 1x128 to 128x1 groups and the weight gradients' scales: how small the 1x128 groups may be.

A column's largest value in 128 rows is at least a code of 2^-9 times a row's scale.  Its scale, the smallest power of two
that takes it to 448 or less, is one that the products take where it is 2^-127 or more: for rows' scales from 2^-110 up
(2^-119 / 448 is above 2^-128), whose groups reach above 448 * 2^-111."""
import numpy as np
import pytest

from oracle import train
import oracle
from _gpu import require_gpu, to_dev, to_host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent,status", [(-109, 0), (-110, 0), (-111, 7), (-127, 7)])
def test_smallest_codes_among_largest(exponent, status):
    torch, fp8bs = require_gpu()
    R = N = K = 128
    q = np.full((R, N), 0x7E, np.uint8)          # 448, and one column of 2^-9
    q[:, 5] = 1
    a = (to_dev(q), torch.full((1, R), 2.0 ** exponent, device="cuda:0"))
    b = (torch.full((R, K), 0x38, dtype=torch.uint8, device="cuda:0"), torch.ones((1, R), device="cuda:0"))
    at, bt = (fp8bs.requant_1x128_to_128x1(*t) for t in (a, b))
    d = fp8bs.grouped_wgrad(*at, *bt, torch.tensor([0, R], dtype=torch.int32, device="cuda:0"))
    assert fp8bs.fp8bs_get_device_status() == status
    if status == 0:
        dec = lambda c, s: oracle.dequantize_1x128(to_host(c), to_host(s).T).astype(np.float64)  # noqa: E731
        ref, mag = train.grouped_wgrad(dec(*at), dec(*bt), [0, R])
        assert np.all(np.abs(to_host(d) - ref) <= 1e-5 * mag) and np.all(to_host(d)[0, 5] > 0)
