"""Rows that belong to no expert: what the grouped products leave there, in front of the first segment and behind the last."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from expert_util import F, MX, O, R, offsets_of, operand, product_tol, spread
from gpu_util import assert_status_ok, require_gpu
from row_util import assert_within, out_tol
from scaled_quantize_gemm_amax_gb300 import linear as L

pytestmark = pytest.mark.gpu
DT = {O.FP32: torch.float32, O.BF16: torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def poisoned(shape, dtype):
    """Gives the allocator a block of this size that holds 9s, which the next allocation of the size takes."""
    t = torch.full(shape, 9.0, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del t


# blocks of the segments, blocks in front and behind, N, K: one CTA a tile, and CTA pairs
CASES = [([1, 0, 2], 2, 1, 256, 256), ([2, 0, 1], 1, 0, 128, 128), ([8, 0, 16, 10] * 6, 3, 2, 2048, 256), ([0, 0], 2, 1, 128, 128)]


@pytest.mark.parametrize("recipe", [R.TENSOR, MX])
@pytest.mark.parametrize("out", [O.BF16, O.FP32])
@pytest.mark.parametrize("blocks,before,behind,n,k", CASES)
def test_the_helper_gives_zeros(blocks, before, behind, n, k, out, recipe):
    starts, offsets = offsets_of(blocks, before)
    cap = starts[-1] + 128 * behind
    q, s, a = operand(spread(cap, k, 1), recipe, F.E4M3)
    qb, sb, b = operand(spread(len(blocks) * n, k, 2), recipe, F.E4M3)
    poisoned((cap, n), DT[out])
    c = fq.grouped_gemm(q, F.E4M3, recipe, s, qb, F.E4M3, recipe, sb, offsets, out=out)
    assert bool((c[:starts[0]] == 0).all()), "in front"
    assert bool((c[starts[-1]:] == 0).all()), "behind"
    for e in range(len(blocks)):
        rows, be = slice(starts[e], starts[e + 1]), b[e * n:(e + 1) * n]
        if rows.start < rows.stop:
            ref = a[rows] @ be.t()
            assert_within(c[rows], ref, out_tol(ref, product_tol(a[rows], be, k, out), DT[out]), f"expert {e}")
    assert_status_ok()


@pytest.mark.parametrize("recipe", [R.TENSOR, MX])
@pytest.mark.parametrize("blocks,before,behind,n,k", CASES)
def test_the_entry_point_leaves_what_it_says(blocks, before, behind, n, k, recipe):
    """0: all rows outside as they were; 1: zeros behind; 2: zeros in front too.  With and without depth."""
    starts, offsets = offsets_of(blocks, before)
    cap = starts[-1] + 128 * behind
    q, s, _ = operand(spread(cap, k, 3), recipe, F.E4M3)
    qb, sb, _ = operand(spread(len(blocks) * n, k, 4), recipe, F.E4M3)
    for depth in (k, 0):
        rows, weights = (q, qb) if depth else (q[:, :0].contiguous(), qb[:, :0].contiguous())
        sa_, sb_ = (s, sb) if depth or recipe == R.TENSOR else (s.new_empty(0), sb.new_empty(0))
        for zero in (0, 1, 2):
            c = torch.full((cap, n), 9.0, dtype=torch.bfloat16, device="cuda")
            fq.fp8_grouped_gemm(rows, F.E4M3, recipe, sa_, weights, F.E4M3, recipe, sb_, offsets, c, zero_tail=zero)
            assert bool((c[:starts[0]] == (0 if zero == 2 else 9)).all()), (depth, zero, "in front")
            assert bool((c[starts[-1]:] == (0 if zero else 9)).all()), (depth, zero, "behind")
            if depth == 0:
                assert bool((c[starts[0]:starts[-1]] == 0).all())
    assert_status_ok()


@pytest.mark.parametrize("recipe", [L.Float8CurrentScaling(), L.MXFP8BlockScaling()])
def test_the_layer_gives_zeros(recipe):
    starts, offsets = offsets_of([1, 2], 2)
    cap = starts[-1] + 128
    layer = L.FP8GroupedLinear(2, 256, 384, device="cuda")
    xs = spread(cap, 256, 5).bfloat16()
    outside = torch.ones(cap, dtype=torch.bool, device="cuda")
    outside[starts[0]:starts[-1]] = False
    xs[outside] = 0
    xs.requires_grad_(True)
    with L.fp8_autocast(fp8_recipe=recipe):
        poisoned((cap, 384), torch.bfloat16)
        y = layer(xs, offsets)
    dy = spread(cap, 384, 6).bfloat16()
    dy[outside] = 0
    poisoned((cap, 256), torch.bfloat16)
    y.backward(dy)
    assert bool((y[outside] == 0).all()) and bool((xs.grad[outside] == 0).all())
    assert bool((y[~outside] != 0).any()) and bool((xs.grad[~outside] != 0).any())
    assert_status_ok()
