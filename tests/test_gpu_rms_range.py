"""RMS norm's gradient of rows far from 1: their factor r is in binary32's range where its square is not."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import assert_status_ok, require_gpu
from row_util import DTYPES, U, assert_within, gen, matrix, out_tol

pytestmark = pytest.mark.gpu

SHAPES = [  # rows, cols, pad, offset: one launch for few rows, 8, 16 and 32 values a lane, rows that registers cannot hold
    (4, 64, 0, 0), (3, 1003, 0, 0), (150, 4096, 0, 0), (400, 256, 0, 0), (400, 1024, 0, 0), (333, 1003, 6, 5), (310, 4099, 0, 0),
    (200, 8200, 0, 0), (170, 9001, 0, 1), (160, 16400, 0, 0), (153, 16401, 0, 0),
]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rms", [1e-20, 3e-15, 5e18])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_gradient_of_rows_far_from_one(rows, cols, pad, offset, rms, dtype):
    dt = DTYPES[dtype]
    h = matrix(rows, cols, dt, 1, pad, offset, rms)
    dy = matrix(rows, cols, dt, 2, 0, 0, 1e-3)
    dy[:, cols // 2:] = 0
    h[0], dy[0] = rms, 0.5      # a projection that is large
    dy[0, ::2] = 0
    w = 1 + 0.2 * torch.randn(cols, generator=gen(3), device="cuda")
    rstd = (1 / h.double().square().mean(1).sqrt()).float()
    assert bool(rstd.isfinite().all())
    dh = (matrix(rows, cols, torch.float32, 4) * rstd[:, None] * 1e-3).to(dt)   # as large as what it is added to
    dx, dw = fq.rms_norm_backward(dy, h, rstd, w, dh=dh)
    r = rstd.double()[:, None]
    xh, g = h.double() * r, dy.double() * w.double()
    c = (g * xh).mean(1, keepdim=True)
    ref = r * (g - xh * c) + dh.double()
    # c: chains of at most 33 products, five additions over a warp and five over the row's, the roundings of g and xh and of the
    # mean: below 48 U of the absolute terms' mean; then a handful of products and sums, each of the magnitude of its terms
    terms = r * g.abs() + r * xh.abs() * c.abs() + dh.double().abs()
    tol = r * xh.abs() * 48 * U * (g * xh).abs().mean(1, keepdim=True) + 8 * U * terms
    assert bool((ref.abs() < torch.finfo(dt).max).all())
    assert_within(dx, ref, out_tol(ref, tol, dt), "dx")
    each = dy.double() * xh
    assert_within(dw, each.sum(0), out_tol(each.sum(0), (rows + 50) * U * each.abs().sum(0), torch.float32), "dweight")
    assert_status_ok()
