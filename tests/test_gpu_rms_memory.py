"""What RMS norm's outputs keep alive: its statistics, which a backward pass holds, not the 8-bit copy beside them."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import require_gpu
from row_util import matrix

pytestmark = pytest.mark.gpu
R = fq.Recipe


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("recipe", [R.TENSOR, R.BLOCK_1x128, R.MX_1x32_TILED])
@pytest.mark.parametrize("keep_y", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_statistics_do_not_hold_the_codes(residual, keep_y, recipe):
    rows, cols = 1024, 2048
    x = matrix(rows, cols, torch.bfloat16, 1)
    res = matrix(rows, cols, torch.bfloat16, 2) if residual else None
    scale = torch.ones(1, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y, h, rstd, q, s = fq.rms_norm(x, None, res, recipe=recipe, scale=scale if recipe == R.TENSOR else None, keep_y=keep_y)
    held = rstd.untyped_storage().nbytes()
    assert held <= (2 * rows * cols if residual else 0) + 4 * rows + 16     # h stays as long as they do
    del y, q, s
    # h, and rstd rounded up to the allocator's 512 bytes
    kept = torch.cuda.memory_allocated() - before
    assert kept <= (2 * rows * cols if residual else 0) + 4 * rows + 512, kept
    assert (h is not None) == residual and rstd.shape == (rows,)
