"""The norm over more rows than its grid holds at once: the ring's stages are filled again and their phases turn.

Per size the rows of a step are at most 152 SMs x 4 CTAs x 8 rows at K = 128, 152 x 4 x 4 at 512 and 1024, 152 x 4 x 2
at 2048, 152 x 4 at 4096, 152 x 2 at 7168 and 152 at 16384 with a residual, so each of these has a third step."""
import numpy as np
import pytest

from oracle import train
from _gpu import require_gpu, to_dev_bf16, to_host
from _train import BF16_HALF, bf16_of, bits_of, check_codes, check_near, f32
from test_norm_gpu import EPS, _gain, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(12000, 128), (5100, 512), (5203, 1024), (2500, 2048), (1301, 4096), (700, 7168), (330, 16384)])
@pytest.mark.parametrize("kind,pow2,residual", [("bf16", True, True), ("f32", False, False), ("f32", True, True), ("bf16", True, False)])
def test_more_rows_than_a_step(M, K, kind, pow2, residual):
    torch, fp8bs = require_gpu()
    x, res = _rows(M, K, 3), _rows(M, K, 4)
    gain, g = _gain(K, kind)
    q, s, y, r, rstd = fp8bs.rmsnorm_quantize(to_dev_bf16(x), gain, to_dev_bf16(res) if residual else None, EPS, pow2, bf16=True)
    rb = bf16_of(f32(x) + f32(res)) if residual else x
    assert np.array_equal(bits_of(r), rb)
    ref, ref_rstd = train.rmsnorm(f32(rb), g, EPS)
    # roundings as counted for fewer rows: they do not depend on the rows
    check_near(to_host(rstd), ref_rstd, ref_rstd, 40, 0.0, "rstd")
    check_near(to_host(y), ref, np.abs(ref), 44, BF16_HALF, "y")
    check_codes(q, s, bits_of(y), pow2, "y")
    assert fp8bs.fp8bs_get_device_status() == 0
