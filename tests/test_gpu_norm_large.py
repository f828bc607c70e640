"""Layer norm's gradient for rows of one large value: mean and rstd are ordinary numbers whose product is
past binary32's range, xh is 0 everywhere, and what a kernel holds past the row's end must not count.
Tolerances as in test_gpu_norm."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import assert_status_ok, require_gpu
from row_util import DTYPES, matrix
from test_gpu_norm import backward_reference, check_backward, params

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("cols", [1, 8, 64, 100, 264, 515, 1003, 1032, 4099, 8200, 12296, 16400])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_of_constant_rows(cols, sign, dtype):
    dt, rows = DTYPES[dtype], 3
    x = torch.full((rows, cols), sign * 2.0 ** 120, dtype=dt, device="cuda")
    mean = torch.full((rows,), sign * 2.0 ** 120, device="cuda")
    rstd = torch.full((rows,), 1e-5 ** -0.5, device="cuda")
    dy, (w, _) = matrix(rows, cols, dt, 560 + cols), params(cols, torch.float32, 14)
    got = fq.layer_norm_backward(dy, rstd, w, x=x, mean=mean)
    assert_status_ok()
    check_backward(got, backward_reference(dy, torch.zeros_like(x, dtype=torch.float64), rstd, w), dt, torch.float32)
