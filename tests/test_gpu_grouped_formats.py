"""Grouped products by formats, exponent rules and multipliers: both operands E4M3 or E5M2, ceil and floor rules mixed, one
multiplier an expert; one CTA a tile and pairs, stacked both ways."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from expert_util import F, MX, O, R, offsets_of, operand, product_tol, spread
from gpu_util import assert_status_ok, require_gpu
from row_util import assert_within, out_tol

pytestmark = pytest.mark.gpu
FLOOR = R.MX_1x32_FLOOR_TILED
RECIPES = [(R.TENSOR, R.TENSOR), (MX, MX), (MX, FLOOR), (FLOOR, MX), (FLOOR, FLOOR)]
FORMATS = [(F.E4M3, F.E4M3), (F.E5M2, F.E4M3), (F.E4M3, F.E5M2), (F.E5M2, F.E5M2)]
# blocks of the segments, N, K: one CTA a tile (per-tensor and MXFP8 at widths of their own), and pairs
CASES = [([2, 0, 1], 384, 384), ([3, 2, 4, 1, 5], 5120, 256)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def widths(recipe, experts, cap, n, m=0):
    return fq.fp8_debug_grouped_plan(recipe, recipe, O.FP32, experts, cap, n, m)["width"]


def test_the_cases_take_both_kernels():
    for recipe in (R.TENSOR, MX):
        (a, n, _), (b, n2, _) = CASES
        assert widths(recipe, len(a), 128 * sum(a), n) > 0 and widths(recipe, len(b), 128 * sum(b), n2) == 0


@pytest.mark.parametrize("stacked", [fq.Stacked.ROWS, fq.Stacked.COLS])
@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("ra,rb", RECIPES)
@pytest.mark.parametrize("blocks,n,k", CASES)
def test_rows(blocks, n, k, ra, rb, fa, fb, stacked):
    starts, offsets = offsets_of(blocks)
    experts, cols = len(blocks), stacked == fq.Stacked.COLS
    q, s, a = operand(spread(starts[-1], k, 1), ra, fa)
    qb, sb, b = operand(spread(n if cols else experts * n, experts * k if cols else k, 2, 3), rb, fb)
    c = fq.grouped_gemm(q, fa, ra, s, qb, fb, rb, sb, offsets, out=O.FP32, stacked=stacked)
    assert_status_ok()
    for e in range(experts):
        rows, be = slice(starts[e], starts[e + 1]), b[:, e * k:(e + 1) * k] if cols else b[e * n:(e + 1) * n]
        if rows.start < rows.stop:
            ref = a[rows] @ be.t()
            assert_within(c[rows], ref, out_tol(ref, product_tol(a[rows], be, k, O.FP32), torch.float32), f"expert {e}")


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("ra,rb", RECIPES)
@pytest.mark.parametrize("m,n", [(384, 128), (768, 4096)])
def test_depth(m, n, ra, rb, fa, fb):
    blocks = [3, 0, 2, 1, 7]
    starts, offsets = offsets_of(blocks)
    q, s, a = operand(spread(m, starts[-1], 3), ra, fa)
    qb, sb, b = operand(spread(n, starts[-1], 4), rb, fb)
    c = fq.grouped_wgrad(q, fa, ra, s, qb, fb, rb, sb, offsets)
    assert_status_ok()
    for e in range(len(blocks)):
        x, y = a[:, starts[e]:starts[e + 1]], b[:, starts[e]:starts[e + 1]]
        ref = x @ y.t()
        assert_within(c[e], ref, out_tol(ref, product_tol(x, y, 128 * blocks[e], O.FP32), torch.float32), f"expert {e}")


@pytest.mark.parametrize("stacked", [fq.Stacked.ROWS, fq.Stacked.COLS])
@pytest.mark.parametrize("out", [O.BF16, O.FP32])
@pytest.mark.parametrize("blocks,n,k", CASES)
def test_a_multiplier_an_expert(blocks, n, k, out, stacked):
    starts, offsets = offsets_of(blocks)
    experts, cols = len(blocks), stacked == fq.Stacked.COLS
    q, s, a = operand(spread(starts[-1], k, 5), R.TENSOR, F.E4M3)
    qb, sb, b = operand(spread(n if cols else experts * n, experts * k if cols else k, 6), R.TENSOR, F.E4M3)
    each = torch.tensor([3.0, 0.25, -7.0, 1e-3, 1.0], device="cuda")[:experts]
    sbe = sb * each
    c = fq.grouped_gemm(q, F.E4M3, R.TENSOR, s, qb, F.E4M3, R.TENSOR, sbe, offsets, out=out, stacked=stacked)
    assert_status_ok()
    dt = torch.float32 if out == O.FP32 else torch.bfloat16
    for e in range(experts):
        rows, be = slice(starts[e], starts[e + 1]), b[:, e * k:(e + 1) * k] if cols else b[e * n:(e + 1) * n]
        if rows.start < rows.stop:
            be = be * (sbe[e].double() / sb[0].double())
            ref = a[rows] @ be.t()
            assert_within(c[rows], ref, out_tol(ref, product_tol(a[rows], be, k, out), dt), f"expert {e}")
