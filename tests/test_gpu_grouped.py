"""Products grouped by expert on the GPU, against 64-bit products of the values that the operands stand for."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from expert_util import F, MX, O, R, offsets_of, operand, product_tol, spread
from gpu_util import Guarded, assert_status_ok, require_gpu
from row_util import assert_within, gen, out_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dt(out):
    return torch.float32 if out == O.FP32 else torch.bfloat16


def _check_rows(c, a, b_of, starts, depth, out, tail):
    """c against every segment's product; rows outside the segments hold `tail` (None: whatever they do)."""
    for e in range(len(starts) - 1):
        rows = slice(starts[e], starts[e + 1])
        if rows.start < rows.stop:
            ref = a[rows] @ b_of(e).t()
            assert_within(c[rows], ref, out_tol(ref, product_tol(a[rows], b_of(e), depth, out), _dt(out)), f"expert {e}")
    if tail is not None:
        assert bool((c[:starts[0]] == tail).all() if starts[0] and tail else True)
        assert bool((c[starts[-1]:] == tail).all())


SHAPES = [  # blocks of 128 rows an expert, blocks before and behind, N, K
    ([1], 0, 0, 128, 128), ([2, 1, 3], 0, 2, 256, 256), ([0, 3, 0, 1, 0], 1, 1, 384, 640), ([1] * 9, 0, 0, 128, 1152),
    ([5, 0, 2], 0, 0, 1280, 384), ([0, 0], 0, 3, 256, 128), ([17], 2, 1, 640, 256), ([1, 2] * 20, 0, 5, 256, 128),
    ([3, 4, 1, 2], 0, 0, 2176, 2048), ([1, 1], 0, 0, 4096, 4096), ([3, 4, 0, 1, 2, 5] * 4, 0, 3, 2176, 384),
    ([1, 9, 0, 6], 1, 2, 10112, 256), ([1], 0, 0, 11008, 256), ([1, 0, 1], 0, 0, 11008, 512), ([1, 1, 1], 0, 0, 11008, 128),
    ([1, 0, 1, 1], 0, 0, 12288, 256), ([2], 1, 1, 9600, 384), ([2, 1, 1], 0, 0, 11008, 256), ([3], 0, 0, 16384, 640),
]


@pytest.mark.parametrize("recipe", [R.TENSOR, MX])
@pytest.mark.parametrize("out", [O.BF16, O.FP32])
@pytest.mark.parametrize("stacked", [fq.Stacked.ROWS, fq.Stacked.COLS])
@pytest.mark.parametrize("blocks,before,behind,n,k", SHAPES)
def test_rows(blocks, before, behind, n, k, stacked, out, recipe):
    starts, offsets = offsets_of(blocks, before)
    experts, cap = len(blocks), starts[-1] + 128 * behind
    fa = F.E5M2 if stacked == fq.Stacked.COLS else F.E4M3
    q, s, a = operand(spread(cap, k, 1), recipe, fa)
    cols = stacked == fq.Stacked.COLS
    qb, sb, b = operand(spread(n if cols else experts * n, experts * k if cols else k, 2, 3) * 0.1, recipe, F.E4M3)
    c = fq.grouped_gemm(q, fa, recipe, s, qb, F.E4M3, recipe, sb, offsets, out=out, stacked=stacked)
    assert c.shape == (cap, n) and c.dtype == _dt(out)
    _check_rows(c, a, lambda e: b[:, e * k:(e + 1) * k] if cols else b[e * n:(e + 1) * n], starts, k, out, 0.0)
    assert_status_ok()


@pytest.mark.parametrize("recipe", [R.TENSOR, MX, R.MX_1x32_FLOOR_TILED])
@pytest.mark.parametrize("out", [O.BF16, O.FP32])
@pytest.mark.parametrize("blocks,before,behind,n,k", SHAPES)
def test_depth(blocks, before, behind, n, k, out, recipe):
    starts, offsets = offsets_of(blocks, before)
    cap = starts[-1] + 128 * behind
    q, s, a = operand(spread(n, cap, 3) * 1e-3, recipe, F.E5M2)
    qb, sb, b = operand(spread(k, cap, 4), recipe, F.E4M3)
    c = fq.grouped_wgrad(q, F.E5M2, recipe, s, qb, F.E4M3, recipe, sb, offsets, out=out)
    assert c.shape == (len(blocks), n, k) and c.dtype == _dt(out)
    for e in range(len(blocks)):
        x, y = a[:, starts[e]:starts[e + 1]], b[:, starts[e]:starts[e + 1]]
        ref = x @ y.t()
        assert_within(c[e], ref, out_tol(ref, product_tol(x, y, 128 * blocks[e], out), _dt(out)), f"expert {e}")
    assert_status_ok()


def test_scales_of_experts():
    """One per-tensor multiplier an expert."""
    starts, offsets = offsets_of([2, 0, 1, 3])
    q, s, a = operand(spread(starts[-1], 256, 5), R.TENSOR, F.E4M3)
    qb, sb, b = operand(spread(4 * 384, 256, 6), R.TENSOR, F.E4M3)
    sb4 = sb * torch.tensor([1.0, 3.0, 0.25, 7.0], device="cuda")
    c = fq.grouped_gemm(q, F.E4M3, R.TENSOR, s, qb, F.E4M3, R.TENSOR, sb4, offsets, out=O.FP32)
    f = [1.0, 3.0, 0.25, 7.0]
    # the multiplier itself is rounded once more: 2 U
    for e in range(4):
        rows = slice(starts[e], starts[e + 1])
        be = b[384 * e:384 * (e + 1)] * f[e]
        ref = a[rows] @ be.t()
        assert_within(c[rows], ref, product_tol(a[rows], be, 256, O.FP32) + 2.0 ** -22 * ref.abs(), f"expert {e}")


@pytest.mark.parametrize("recipe", [R.TENSOR, MX])
@pytest.mark.parametrize("out", [O.BF16, O.FP32])
def test_outputs_stay_inside(out, recipe):
    """Guards around the output; rows outside the segments as they were, or zeros behind the last."""
    starts, offsets = offsets_of([3, 0, 2], 1)
    cap, n, k = starts[-1] + 256, 384, 256
    q, s, a = operand(spread(cap, k, 7), recipe, F.E4M3)
    qb, sb, b = operand(spread(3 * n, k, 8), recipe, F.E4M3)
    for zero in (False, True):
        g = Guarded((cap, n), _dt(out))
        was = g.t.clone()
        fq.fp8_grouped_gemm(q, F.E4M3, recipe, s, qb, F.E4M3, recipe, sb, offsets, g.t, out, zero_tail=zero)
        g.check("c")
        raw, old = g.t.view(torch.uint8), was.view(torch.uint8)
        assert torch.equal(raw[:128], old[:128])
        assert bool((g.t[starts[-1]:] == 0).all()) if zero else torch.equal(raw[starts[-1]:], old[starts[-1]:])
        _check_rows(g.t, a, lambda e: b[e * n:(e + 1) * n], starts, k, out, None)
    qc, sc, _ = operand(spread(n, cap, 9), recipe, F.E4M3)
    qd, sd, _ = operand(spread(256, cap, 10), recipe, F.E4M3)
    g = Guarded((3, n, 256), _dt(out))
    fq.fp8_grouped_wgrad(qc, F.E4M3, recipe, sc, qd, F.E4M3, recipe, sd, offsets, g.t, out)
    g.check("dw")
    assert torch.equal(g.t, fq.grouped_wgrad(qc, F.E4M3, recipe, sc, qd, F.E4M3, recipe, sd, offsets, out=out))
    assert bool((g.t[1] == 0).all())
    assert_status_ok()


@pytest.mark.parametrize("bad", [[0, 100, 256], [0, 256, 128], [-128, 128, 256], [0, 128, 640], [0, 256, 2 ** 31 - 128], [64, 192, 320]])
def test_bad_offsets(bad):
    """Offsets that are not ascending multiples of 128 within the capacity write nothing and are reported."""
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
    q, s, _ = operand(spread(512, 128, 11), MX, F.E4M3)
    qb, sb, _ = operand(spread(2 * 128, 128, 12), MX, F.E4M3)
    c = torch.full((512, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8_grouped_gemm(q, F.E4M3, MX, s, qb, F.E4M3, MX, sb, offsets, c, zero_tail=True)
    assert fq.fp8_get_device_status() == fq.Status.ERR_DEVICE_STATE
    assert bool((c == 7).all())
    qc, sc, _ = operand(spread(128, 512, 13), MX, F.E4M3)
    d = torch.full((2, 128, 128), 7.0, device="cuda")
    fq.fp8_grouped_wgrad(qc, F.E4M3, MX, sc, qc, F.E4M3, MX, sc, offsets, d)
    assert fq.fp8_get_device_status() == fq.Status.ERR_DEVICE_STATE
    assert bool((d == 7).all())
    assert_status_ok()


def test_empty():
    _, offsets = offsets_of([0, 0, 0])
    one = torch.ones(1, device="cuda")
    z = torch.empty((0, 256), dtype=torch.uint8, device="cuda")
    w = torch.zeros((3 * 128, 256), dtype=torch.uint8, device="cuda")
    assert fq.grouped_gemm(z, F.E4M3, R.TENSOR, one, w, F.E4M3, R.TENSOR, one, offsets).shape == (0, 128)
    zc = torch.empty((128, 0), dtype=torch.uint8, device="cuda")
    dw = fq.grouped_wgrad(zc, F.E4M3, R.TENSOR, one, zc, F.E4M3, R.TENSOR, one, offsets)
    assert dw.shape == (3, 128, 128) and bool((dw == 0).all())
    # no depth: the segments' rows are 0, the others as they were
    starts, some = offsets_of([1, 0, 1])
    c = torch.full((512, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    fq.fp8_grouped_gemm(torch.empty((512, 0), dtype=torch.uint8, device="cuda"), F.E4M3, R.TENSOR, one,
                        torch.empty((3 * 128, 0), dtype=torch.uint8, device="cuda"), F.E4M3, R.TENSOR, one, some, c)
    assert bool((c[:256] == 0).all()) and bool((c[256:] == 3).all())
    assert_status_ok()


def test_many_experts():
    """1024 experts, most without rows."""
    blocks = [1 if e % 37 == 5 else 0 for e in range(1024)]
    starts, offsets = offsets_of(blocks)
    q, s, a = operand(spread(starts[-1], 128, 14), MX, F.E4M3)
    qb, sb, b = operand(spread(1024 * 128, 128, 15), MX, F.E4M3)
    c = fq.grouped_gemm(q, F.E4M3, MX, s, qb, F.E4M3, MX, sb, offsets, out=O.FP32)
    _check_rows(c, a, lambda e: b[128 * e:128 * (e + 1)], starts, 128, O.FP32, None)
    assert_status_ok()


def test_many_experts_of_many_rows():
    """More experts than the deepest ring of stages leaves room for."""
    blocks = [(e * 7) % 4 for e in range(260)]
    starts, offsets = offsets_of(blocks)
    q, s, a = operand(spread(starts[-1], 256, 20), R.TENSOR, F.E4M3)
    qb, sb, b = operand(spread(260 * 256, 256, 21), R.TENSOR, F.E4M3)
    c = fq.grouped_gemm(q, F.E4M3, R.TENSOR, s, qb, F.E4M3, R.TENSOR, sb, offsets, out=O.FP32)
    _check_rows(c, a, lambda e: b[256 * e:256 * (e + 1)], starts, 256, O.FP32, None)
    assert_status_ok()


def test_two_at_once_and_captured():
    """The routing made inside a captured graph, replayed for another one; two calls on two streams at once."""
    tokens, k, experts, cols, n = 200, 2, 5, 256, 384
    ids = torch.randint(0, experts, (tokens, k), generator=gen(16), device="cuda")
    x = torch.randn((tokens, cols), generator=gen(17), device="cuda").bfloat16()
    qb, sb, _ = operand(spread(experts * n, cols, 18), MX, F.E4M3)

    def step():
        route = fq.moe_route(ids, experts, align=128)
        q, s, _, _ = fq.cast_transpose(fq.moe_dispatch(x, route), MX, F.E4M3, col=False)
        y = fq.grouped_gemm(q, F.E4M3, MX, s, qb, F.E4M3, MX, sb, route.offsets)
        return fq.moe_combine(y, route)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    ids.copy_(torch.where(torch.rand((tokens, k), generator=gen(19), device="cuda") < 0.7, 3, ids))
    want = step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs.append([step() for _ in range(3)])
    torch.cuda.synchronize()
    for one in outs:
        for y in one:
            assert torch.equal(y, want)
    assert_status_ok()
