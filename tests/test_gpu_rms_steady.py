"""RMS norm where every group of warps works on many rows: stages refilled, buffers in turn, several sweeps of the largest grid.
The numbers of rows follow from the GPU's SMs; the tolerances from the chains of sums at each width."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
import test_gpu_rms as rms
from expert_util import F, R, e8m0_values, values
from gpu_util import assert_status_ok, require_gpu
from row_util import DTYPES, FMAX, U, assert_within, gen, matrix, out_tol

pytestmark = pytest.mark.gpu
EPS = 1e-5
TURNS = 9        # rows of a group: more than twice the stages in flight (4 at most), and one


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rows_for(cols):
    """Rows that give every group TURNS of them: a block an SM, as many groups as 32 warps can be at most."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if cols > 16384:
        return sms * 8 * 3 + 5      # blocks that take one row after another, eight an SM
    lane = 8 if cols <= 256 else 16     # the fewest values a lane: the most warps a row, so never fewer groups than there are
    warps = -(-cols // (32 * (lane if cols <= 512 else 32)))
    return sms * max(1, (32 if cols <= 256 else 24) // warps) * TURNS + 5


def r_tol(cols):
    """1 / sqrt(mean): a lane's 8 to 32 squares in two chains, one addition, five over the warp, five over the row's warps, 1 / n and
    eps: V / 2 + 13 U of the mean; wider rows cols / 512 of a thread in one chain, five and 16 additions.  The root halves that; the
    reciprocal root, its step and the two products behind it add less than 8 U."""
    return ((cols / 512 + 24 if cols > 16384 else 29) / 2 + 8) * U


# a warp a row (8, 16 and 32 values a lane), several, the widest, wider; odd and even, aligned and not
WIDTHS = [96, 128, 250, 256, 400, 512, 1000, 1024, 1003, 2560, 3001, 4096, 4099, 5120, 8192, 8200, 9001, 12288, 12301, 16381, 16384, 16400,
          20001]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward(cols, residual, dtype):
    rows, dt, pad = rows_for(cols), DTYPES[dtype], 8 if cols % 64 == 0 else 0
    x = matrix(rows, cols, dt, 1, pad, 0, 3.0)
    res = matrix(rows, cols, dt, 2, 0, 0, 2.0) if residual else None
    w = rms._weight(cols, torch.float32, 3)
    y, h, rstd, _, _ = fq.rms_norm(x, w, res, EPS)
    assert_status_ok()
    h64, r64, y64 = rms._exact(x, res, w)
    if residual:
        assert torch.equal(h.double(), h64)
    assert_within(rstd, r64, r_tol(cols) * r64, "rstd")
    assert_within(y, y64, out_tol(y64, r_tol(cols) * y64.abs(), dt), "y")


CODES = [(R.TENSOR, 250), (R.BLOCK_1x128, 128), (R.MX_1x32, 96), (R.MX_1x32_TILED, 256), (R.BLOCK_1x128, 400), (R.MX_1x32_FLOOR, 512),
         (R.TENSOR, 1003), (R.BLOCK_1x128, 1003), (R.MX_1x32, 1056), (R.MX_1x32_TILED, 1024), (R.BLOCK_1x128, 4096), (R.TENSOR, 4096),
         (R.MX_1x32_TILED, 4096), (R.MX_1x32_FLOOR_TILED, 8192), (R.BLOCK_1x128, 4099), (R.BLOCK_1x128, 12301), (R.MX_1x32, 12288),
         (R.MX_1x32_TILED, 16384), (R.TENSOR, 16400), (R.BLOCK_1x128, 20001), (R.MX_1x32_TILED, 16512)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("recipe,cols", CODES)
def test_codes(recipe, cols, dtype):
    """With binary32 data the bytes of the library's cast of y; else within half a step of the exact value."""
    dt, fmt = DTYPES[dtype], F.E4M3
    tiled = recipe in (R.MX_1x32_TILED, R.MX_1x32_FLOOR_TILED)
    rows = rows_for(cols) if cols % 128 else (rows_for(cols) + 127) // 128 * 128
    x, res, w = matrix(rows, cols, dt, 5, 0, 0, 3.0), matrix(rows, cols, dt, 6), rms._weight(cols, torch.float32, 7)
    scale = torch.full((1,), FMAX[int(fmt)] / 8.0, device="cuda") if recipe == R.TENSOR else None
    amax = torch.full((1,), 9e9, device="cuda") if recipe == R.TENSOR else None
    y, h, rstd, q, s = fq.rms_norm(x, w, res, EPS, recipe=recipe, fmt=fmt, scale=scale, amax_out=amax)
    assert_status_ok()
    h64, r64, y64 = rms._exact(x, res, w)
    assert torch.equal(h.double(), h64)
    tol = r_tol(cols)
    if recipe == R.TENSOR:
        assert_within(amax, y64.abs().max().reshape(1), tol * y64.abs().max().reshape(1), "amax")
        mult = s.double().expand(rows, cols)
    elif recipe == R.BLOCK_1x128:
        a = torch.stack([p.abs().amax(1) for p in y64.split(128, 1)], 1)
        assert_within(s, a / FMAX[int(fmt)], (tol + 3 * U) * a / FMAX[int(fmt)], "multipliers")
        mult = s.double().repeat_interleave(128, 1)[:, :cols]
    else:
        mult = e8m0_values(s, rows, cols, tiled).repeat_interleave(32, 1)
        a = y64.view(rows, -1, 32).abs().amax(2)
        floor = recipe in (R.MX_1x32_FLOOR, R.MX_1x32_FLOOR_TILED)
        e = torch.floor(torch.log2(a)) - 8
        if not floor:
            e = e + (a / torch.exp2(e + 8) > 1.75)
        assert bool(((mult[:, ::32] == torch.exp2(e)) | rms._near_border(a, fmt, floor)).all())
    if dtype == "fp32" and cols % 128 == 0:
        qc, sc, _, _ = fq.cast_transpose(y, recipe, fmt, scale, col=False)
        assert torch.equal(q, qc) and (recipe == R.TENSOR or torch.equal(s.view(torch.uint8), sc.view(torch.uint8)))
    ref = y64.clamp(-448 * mult, 448 * mult)
    assert_within(values(q, recipe, fmt, s), ref, y64.abs() * (2.0 ** -4 + 2 * tol) + 2.0 ** -10 * mult * (1 + 1e-6), "codes")
    only = fq.rms_norm(x, w, res, EPS, recipe=recipe, fmt=fmt, scale=scale, keep_y=False, stats=False)
    assert torch.equal(only[1], h) and torch.equal(only[3], q) and torch.equal(only[4].view(torch.uint8), s.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("cols", WIDTHS)
def test_backward(cols, stream, dtype):
    rows, dt, pad = rows_for(cols), DTYPES[dtype], 8 if cols % 64 == 0 else 0
    h, dy = matrix(rows, cols, dt, 21, pad, 0, 3.0), matrix(rows, cols, dt, 22, 0, 0, 1e-2)
    dh = matrix(rows, cols, dt, 23, 0, 0, 1e-2) if stream else None
    w = rms._weight(cols, torch.float32, 24)
    rstd = 1 / (h.float().square().mean(1) + EPS).sqrt()
    dx, dw = fq.rms_norm_backward(dy, h, rstd, w, dh=dh)
    assert_status_ok()
    r = rstd.double()[:, None]
    xh, g = h.double() * r, dy.double() * w.double()
    c = (g * xh).mean(1, keepdim=True)
    add = 0.0 if dh is None else dh.double()
    ref = r * (g - xh * c) + add
    # c: at most 40 products in a chain, ten more additions, the roundings of g and xh and of the mean: below 56 U of the terms' mean
    tol = r * xh.abs() * 56 * U * (g * xh).abs().mean(1, keepdim=True) + 8 * U * (r * g.abs() + r * (xh * c).abs())
    tol = tol + (0.0 if dh is None else 8 * U * dh.double().abs())
    assert_within(dx, ref, out_tol(ref, tol, dt), "dx")
    del ref, tol, add
    terms = dy.double() * xh
    # a group's rows in one chain (up to a wave of rows an SM in rows that registers cannot hold), its block's groups, the partial sums
    total, size = terms.sum(0), terms.abs().sum(0)
    assert_within(dw, total, out_tol(total, (rows / 32 + 128) * U * size, torch.float32), "dweight")
    again = fq.rms_norm_backward(dy, h, rstd, w, dh=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_the_same_bits_every_time():
    for cols in (250, 1003, 4096, 5120, 12288):
        rows = rows_for(cols)
        x, res = matrix(rows, cols, torch.bfloat16, 31), matrix(rows, cols, torch.bfloat16, 32)
        first = None
        for _ in range(3):
            out = [t for t in fq.rms_norm(x, None, res, EPS, recipe=R.BLOCK_1x128) if t is not None]
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, out))
            first = out
    assert_status_ok()
