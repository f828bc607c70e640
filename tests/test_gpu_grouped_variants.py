"""Every kernel, ring and tile width of the grouped products, on walks of several tiles a CTA, against 64-bit products."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from expert_util import F, offsets_of, operand, product_tol, spread
from gpu_util import assert_status_ok, require_gpu
from grouped_cases import DEPTH, MX, O, ROWS, segments
from row_util import assert_within, out_tol

pytestmark = pytest.mark.gpu
DT = {O.FP32: torch.float32, O.BF16: torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def taken(recipe, out, experts, capacity, n, m, width):
    """The case takes the form it is here for, if this GPU has the SMs that the cases are written for."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 152:
        assert fq.fp8_debug_grouped_plan(recipe, recipe, out, experts, capacity, n, m, sms)["width"] == width


@pytest.mark.parametrize("out", [O.BF16, O.FP32])
@pytest.mark.parametrize("recipe,experts,blocks,n,k,width,stages,third", ROWS)
def test_rows(recipe, experts, blocks, n, k, width, stages, third, out):
    segs = segments(experts, blocks)
    starts, offsets = offsets_of(segs)
    taken(recipe, out, experts, starts[-1], n, 0, width)
    q, s, a = operand(spread(starts[-1], k, 1), recipe, F.E4M3)
    qb, sb, b = operand(spread(experts * n, k, 2, 3), recipe, F.E4M3)
    c = fq.grouped_gemm(q, F.E4M3, recipe, s, qb, F.E4M3, recipe, sb, offsets, out=out)
    assert_status_ok()
    ref, tol = torch.zeros(starts[-1], n, dtype=torch.float64, device="cuda"), torch.zeros(starts[-1], n, dtype=torch.float64, device="cuda")
    for e in range(experts):
        if segs[e]:
            rows, be = slice(starts[e], starts[e + 1]), b[e * n:(e + 1) * n]
            ref[rows], tol[rows] = a[rows] @ be.t(), product_tol(a[rows], be, k, out)
    assert_within(c, ref, out_tol(ref, tol, DT[out]), "c")


@pytest.mark.parametrize("out", [O.BF16, O.FP32])
@pytest.mark.parametrize("recipe,experts,blocks,m,n,width,stages,third", DEPTH)
def test_depth(recipe, experts, blocks, m, n, width, stages, third, out):
    segs = segments(experts, blocks)
    starts, offsets = offsets_of(segs)
    taken(recipe, out, experts, starts[-1], n, m, width)
    fmt = F.E5M2 if recipe == MX else F.E4M3
    q, s, a = operand(spread(m, starts[-1], 3), recipe, fmt)
    qb, sb, b = operand(spread(n, starts[-1], 4), recipe, F.E4M3)
    c = fq.grouped_wgrad(q, fmt, recipe, s, qb, F.E4M3, recipe, sb, offsets, out=out)
    assert_status_ok()
    ref, tol = torch.zeros(c.shape, dtype=torch.float64, device="cuda"), torch.zeros(c.shape, dtype=torch.float64, device="cuda")
    for e in range(experts):
        x, y = a[:, starts[e]:starts[e + 1]], b[:, starts[e]:starts[e + 1]]
        ref[e], tol[e] = x @ y.t(), product_tol(x, y, 128 * segs[e], out)
    assert_within(c, ref, out_tol(ref, tol, DT[out]), "dw")


@pytest.mark.parametrize("out", [O.BF16, O.FP32])
@pytest.mark.parametrize("recipe,experts,blocks,n,k,width,stages,third", [c for c in ROWS if c[-1]])
def test_the_same_bits_every_time(recipe, experts, blocks, n, k, width, stages, third, out):
    """Stacked the other way, from other calls and in a graph beside another stream's: what a CTA's earlier tiles left is not in it."""
    segs = segments(experts, blocks)
    starts, offsets = offsets_of(segs)
    q, s, _ = operand(spread(starts[-1], k, 5), recipe, F.E4M3)
    w = spread(experts * n, k, 6, 3)
    qb, sb, _ = operand(w, recipe, F.E4M3)
    side_by_side = w.view(experts, n, k).transpose(0, 1).reshape(n, experts * k)
    qc, sc, _ = operand(side_by_side, recipe, F.E4M3)
    rows = lambda: fq.grouped_gemm(q, F.E4M3, recipe, s, qb, F.E4M3, recipe, sb, offsets, out=out)   # noqa: E731
    first = rows()
    cols = fq.grouped_gemm(q, F.E4M3, recipe, s, qc, F.E4M3, recipe, sc, offsets, out=out, stacked=fq.Stacked.COLS)
    assert torch.equal(cols, first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [rows() for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g.replay()
    with torch.cuda.stream(side):
        beside = [rows() for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(c, first) for c in got + beside)
    assert_status_ok()
