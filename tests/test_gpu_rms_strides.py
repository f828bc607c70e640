"""RMS norm into matrices with row strides and starts of their own: the values, and nothing written between the rows."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from expert_util import F, R, e8m0_values, values
from gpu_util import assert_status_ok, require_gpu
from row_util import DTYPES, U, assert_within, gen, matrix, out_tol
from test_gpu_rms_steady import r_tol

pytestmark = pytest.mark.gpu
EPS = 1e-5
SENTINEL = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Strided:
    """A matrix with `pad` elements behind every row and `offset` in front of the first, all of it filled with one byte."""

    def __init__(self, rows, cols, dtype, pad, offset):
        self.buf = torch.empty(offset + rows * (cols + pad) + 64, dtype=dtype, device="cuda")
        self.buf.view(torch.uint8).fill_(SENTINEL)
        self.inside = torch.zeros(self.buf.numel(), dtype=torch.bool, device="cuda")
        place = slice(offset, offset + rows * (cols + pad))
        self.t = self.buf[place].view(rows, cols + pad)[:, :cols]
        self.inside[place].view(rows, cols + pad)[:, :cols] = True

    def check(self, what):
        outside = self.buf.view(torch.uint8).view(self.buf.numel(), -1)[~self.inside]
        assert bool((outside == SENTINEL).all()), f"{what}: written outside its rows"


# of x, residual, h, y, codes, dy, dh, dx: pads and offsets; all at 16 bytes, each at another place, one alone off
LAYOUTS = {
    "aligned": [(16, 16), (32, 0), (16, 48), (48, 16), (16, 16), (0, 32), (16, 0), (64, 16)],
    "mixed": [(1, 3), (6, 0), (3, 5), (2, 1), (5, 7), (8, 8), (0, 1), (7, 2)],
    "y off": [(0, 0), (16, 0), (16, 0), (1, 1), (16, 0), (16, 0), (0, 0), (3, 1)],
    "codes off": [(0, 0), (0, 0), (0, 0), (0, 0), (3, 1), (0, 0), (1, 0), (0, 0)],
}
SHAPES = [(1, 4096), (3, 1003), (150, 1024), (200, 256), (333, 96), (400, 4096), (310, 4099), (155, 8200), (160, 16400), (153, 16401)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(rows, cols, layout, dtype):
    dt, at = DTYPES[dtype], LAYOUTS[layout]
    inputs = [matrix(rows, cols, dt, 1 + i, *at[j], 3.0 - i) for i, j in ((0, 0), (1, 1))]
    x, res = inputs
    dy, dh = matrix(rows, cols, dt, 5, *at[5], 1e-2), matrix(rows, cols, dt, 6, *at[6], 1e-2)
    w = 1 + 0.2 * torch.randn(cols, generator=gen(7), device="cuda")
    h, y, q, dx = (Strided(rows, cols, t, *at[j]) for t, j in ((dt, 2), (dt, 3), (torch.uint8, 4), (dt, 7)))
    rstd, dw = torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda")
    mx = cols % 32 == 0
    s = torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda") if mx else torch.empty((rows, -(-cols // 128)), device="cuda")
    recipe = R.MX_1x32 if mx else R.BLOCK_1x128
    fq.fp8_rms_norm(x, res, w, EPS, h.t, y.t, rstd, recipe, F.E4M3, None, None, q.t, s)
    ws = torch.empty(fq.fp8_rms_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    fq.fp8_rms_norm_backward(dy, h.t, rstd, dh, w, dx.t, dw, ws)
    assert_status_ok()
    for m, what in ((h, "h"), (y, "y"), (q, "codes"), (dx, "dx")):
        m.check(what)
    h64 = (x.float() + res.float()).to(dt).double()
    assert torch.equal(h.t.double(), h64)
    r64 = 1 / (h64.square().mean(1) + EPS).sqrt()
    y64, tol = h64 * r64[:, None] * w.double(), r_tol(cols)
    assert_within(rstd, r64, tol * r64, "rstd")
    assert_within(y.t, y64, out_tol(y64, tol * y64.abs(), dt), "y")
    mult = e8m0_values(s, rows, cols, False).repeat_interleave(32, 1) if mx else s.double().repeat_interleave(128, 1)[:, :cols]
    assert_within(values(q.t, recipe, F.E4M3, s), y64.clamp(-448 * mult, 448 * mult),
                  y64.abs() * (2.0 ** -4 + 2 * tol) + 2.0 ** -10 * mult * (1 + 1e-6), "codes")
    r = rstd.double()[:, None]
    xh, g = h64 * r, dy.double() * w.double()
    c = (g * xh).mean(1, keepdim=True)
    ref = r * (g - xh * c) + dh.double()
    # as in the tests of many rows: c below 56 U of the terms' mean, a handful of products and sums behind it
    tol = r * xh.abs() * 56 * U * (g * xh).abs().mean(1, keepdim=True) + 8 * U * (r * g.abs() + r * (xh * c).abs() + dh.double().abs())
    assert_within(dx.t, ref, out_tol(ref, tol, dt), "dx")
    terms = dy.double() * xh
    assert_within(dw, terms.sum(0), out_tol(terms.sum(0), (rows / 16 + 128) * U * terms.abs().sum(0), torch.float32), "dweight")
