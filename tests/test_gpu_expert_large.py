"""RMS norm, grouped products and gradient clipping where places in memory pass 32 bits."""
import math

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
import test_gpu_rms as rms
from expert_util import F, MX, O, R, offsets_of, operand, product_tol, spread
from gpu_util import assert_status_ok, require_gpu
from row_util import BF16, U, assert_within, gen, out_tol

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def large(rows, cols, seed, dtype=torch.bfloat16, sigma=1.0):
    """[rows, cols] normal values, made a part at a time."""
    v = torch.empty((rows, cols), dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // cols)
    for i in range(0, rows, step):
        v[i:i + step] = torch.randn((min(step, rows - i), cols), generator=gen(seed + i), device="cuda") * sigma
    return v


# rows and columns whose product passes 2^31 elements: many narrow rows, ordinary ones, odd ones, the widest
@pytest.mark.parametrize("rows,cols", [(17_000_000, 128), (540_000, 4096), (530_000, 4099), (135_000, 16384), (110_000, 20001)])
def test_rms(rows, cols):
    x, res = large(rows, cols, 1, sigma=3.0), large(rows, cols, 7)
    w = rms._weight(cols, torch.float32, 3)
    recipe = R.BLOCK_1x128
    y, h, rstd, q, s = fq.rms_norm(x, w, res, EPS, recipe=recipe)
    dx, dw = fq.rms_norm_backward(x, h, rstd, w, dh=res)
    assert_status_ok()
    for i in (0, 1 + (1 << 31) // cols - 1000, rows - 1500):      # at the start, around the border and at the end
        part = slice(max(i, 0), min(max(i, 0) + 1500, rows))
        h64, r64, y64 = rms._exact(x[part], res[part], w)
        assert torch.equal(h[part].double(), h64)
        assert_within(rstd[part], r64, rms.R_TOL * r64, "rstd")
        assert_within(y[part], y64, out_tol(y64, rms.R_TOL * y64.abs(), torch.bfloat16), "y")
        small = fq.rms_norm(x[part], w, res[part], EPS, recipe=recipe)
        mult = s[part].double().repeat_interleave(128, 1)[:, :cols]
        code = q[part].contiguous().view(torch.float8_e4m3fn).double() * mult
        assert_within(code, y64.clamp(-448 * mult, 448 * mult), y64.abs() * (2.0 ** -4 + 2 * rms.R_TOL) + 2.0 ** -10 * mult * (1 + 1e-6),
                      "codes")
        again, _ = fq.rms_norm_backward(x[part], small[1], rstd[part], w, dh=res[part])
        r = rstd[part].double()[:, None]
        xh, g = h64 * r, x[part].double() * w.double()
        c = (g * xh).mean(1, keepdim=True)
        ref = r * (g - xh * c) + res[part].double()
        tol = r * xh.abs() * 56 * U * (g * xh).abs().mean(1, keepdim=True) + 8 * U * (r * g.abs() + r * (xh * c).abs() + res[part].double().abs())
        assert_within(dx[part], ref, out_tol(ref, tol, torch.bfloat16), "dx")
        assert_within(again, ref, out_tol(ref, tol, torch.bfloat16), "dx of the part")
    total, size = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 20_000_000 // cols + 1):
        part = slice(i, i + 20_000_000 // cols + 1)
        terms = x[part].double() * (h[part].double() * rstd[part].double()[:, None])
        total += terms.sum(0)
        size += terms.abs().sum(0)
    # chains of the rows of a group, 152 blocks of one group at least
    assert_within(dw, total, (rows / 152 + 128) * U * size, "dweight")


@pytest.mark.parametrize("recipe", [R.TENSOR, MX])
@pytest.mark.parametrize("out", [O.BF16, O.FP32])
def test_grouped(out, recipe):
    """An output of more than 2^31 elements."""
    dt = torch.float32 if out == O.FP32 else torch.bfloat16
    n, k, experts = 4096, 128, 5
    blocks = [900, 0, 1401, 1, 1900]
    starts, offsets = offsets_of(blocks)
    cap = starts[-1] + 128
    assert cap * n > 2 ** 31
    q, s, a = operand(spread(cap, k, 1), recipe, F.E4M3)
    qb, sb, b = operand(spread(experts * n, k, 2, 3), recipe, F.E4M3)
    c = fq.grouped_gemm(q, F.E4M3, recipe, s, qb, F.E4M3, recipe, sb, offsets, out=out)
    assert_status_ok()
    for e in range(experts):
        for lo in {starts[e], max(starts[e], starts[e + 1] - 1024)}:
            rows = slice(lo, min(lo + 1024, starts[e + 1]))
            if rows.start < rows.stop:
                be = b[e * n:(e + 1) * n]
                ref = a[rows] @ be.t()
                assert_within(c[rows], ref, out_tol(ref, product_tol(a[rows], be, k, out), dt), f"expert {e} at {lo}")
    assert bool((c[starts[-1]:] == 0).all())


@pytest.mark.parametrize("recipe", [R.TENSOR, MX])
def test_grouped_weights(recipe):
    m, n, experts = 4096, 4096, 130
    assert experts * m * n > 2 ** 31
    segs = [e % 3 for e in range(experts)]
    starts, offsets = offsets_of(segs)
    q, s, a = operand(spread(m, starts[-1], 3), recipe, F.E4M3)
    qb, sb, b = operand(spread(n, starts[-1], 4), recipe, F.E4M3)
    c = fq.grouped_wgrad(q, F.E4M3, recipe, s, qb, F.E4M3, recipe, sb, offsets)
    assert_status_ok()
    for e in (0, 1, 2, 126, 127, 128, 129):
        x, y = a[:, starts[e]:starts[e + 1]], b[:, starts[e]:starts[e + 1]]
        ref = x @ y.t()
        assert_within(c[e], ref, out_tol(ref, product_tol(x, y, 128 * segs[e], O.FP32), torch.float32), f"expert {e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_clip(dtype):
    """One gradient of more than 2^32 elements beside small ones, at an odd place."""
    n = 2 ** 32 + 12345 if dtype == torch.bfloat16 else 2 ** 31 + 12345
    buf = torch.empty(n + 3, dtype=dtype, device="cuda")
    step = 1 << 28
    for i in range(0, n + 3, step):
        buf[i:i + step] = torch.randn(min(step, n + 3 - i), generator=gen(i % 1000003), device="cuda")
    grads = [torch.ones(77, dtype=dtype, device="cuda"), buf[3:], torch.ones(5, device="cuda")]
    ref = math.fsum(float(g[i:i + step].double().square().sum()) for g in grads for i in range(0, g.numel(), step)) ** 0.5
    front = buf[:3].clone()
    was = [(i, grads[1][i:i + 5000].clone()) for i in (0, 2 ** 31 - 2500, n - 5000)]
    norm = fq.clip_grad_norm(grads, 100.0)
    assert abs(float(norm) - ref) <= 10 * U * ref
    by = 100.0 / (ref + 1e-6)
    half = BF16 if dtype == torch.bfloat16 else U
    for i, w in was:
        want = w.double() * by
        assert bool(((grads[1][i:i + 5000].double() - want).abs() <= want.abs() * (14 * U + half) + 2.0 ** -133).all()), i
    assert torch.equal(buf[:3], front)
    after = math.fsum(float(g[i:i + step].double().square().sum()) for g in grads for i in range(0, g.numel(), step)) ** 0.5
    assert abs(after - 100.0) <= 100.0 * half
