"""RMS norm on the GPU: outputs and gradients against 64-bit formulas, the 8-bit outputs against the library's own cast
and the codes' error bound, at widths, strides, alignments and sizes where the kernels' variants meet."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from expert_util import F, R, e8m0_values, values
from gpu_util import Guarded, assert_status_ok, require_gpu
from row_util import BF16, DTYPES, FMAX, TINY, U, assert_within, gen, matrix, out_tol

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _exact(x, res, w, eps=EPS):
    h = x.double() if res is None else (x.float() + res.float()).to(x.dtype).double()
    r = 1 / (h.square().mean(1) + eps).sqrt()
    return h, r, h * r[:, None] * (1.0 if w is None else w.double())


# The sum of squares has relative error at most (V / 2 + 10) U with V = 32 values a lane, (cols / 256 + 13) U in rows of more than
# 16384 columns: at most 93 U at 20480.  Its root halves that; the reciprocal root, its step and two products add less than 8 U.
R_TOL = 55 * U


def _weight(cols, dtype, seed):
    return (1 + 0.2 * torch.randn(cols, generator=gen(seed), device="cuda")).to(dtype)


CASES = [  # rows, cols, pad, offset
    (1, 4096, 0, 0), (1, 1, 0, 0), (3, 8, 0, 0), (5, 7, 3, 1), (33, 128, 0, 0), (37, 250, 6, 0), (300, 256, 0, 0), (129, 384, 8, 8),
    (41, 511, 1, 3), (160, 512, 0, 0), (17, 1000, 0, 0), (700, 1024, 0, 0), (31, 1003, 6, 5), (9, 4099, 0, 0), (457, 4096, 16, 0),
    (6, 8192, 0, 0), (3, 12288, 0, 0), (2, 16383, 0, 1), (2, 16384, 0, 0), (3, 16392, 0, 0), (2, 20480, 0, 0), (305, 2048, 0, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols,pad,offset", CASES)
def test_forward(rows, cols, pad, offset, residual, dtype):
    dt = DTYPES[dtype]
    x = matrix(rows, cols, dt, 1, pad, offset, 3.0)
    res = matrix(rows, cols, dt, 2, pad // 2, offset, 2.0) if residual else None
    w = _weight(cols, torch.bfloat16 if rows % 2 else torch.float32, 3) if cols != 1024 else None
    y, h, rstd, q, s = fq.rms_norm(x, w, res, EPS)
    h64, r64, y64 = _exact(x, res, w)
    assert q is None and s is None
    if residual:
        assert torch.equal(h.double(), h64)
    else:
        assert h is None
    assert_within(rstd, r64, R_TOL * r64, "rstd")
    assert_within(y, y64, out_tol(y64, R_TOL * y64.abs(), dt), "y")


RECIPES = [R.TENSOR, R.BLOCK_1x128, R.MX_1x32, R.MX_1x32_FLOOR, R.MX_1x32_TILED, R.MX_1x32_FLOOR_TILED]


def _near_border(amax, fmt, floor):
    """Blocks whose exact amax lies so near a border of the exponent rule that binary32 may fall on its other side."""
    m = amax / torch.exp2(torch.floor(torch.log2(amax.clamp(min=1e-300))))
    b = torch.tensor([1.0, 2.0] if floor else [1.75], dtype=torch.float64, device="cuda")
    return ((m[..., None] - b).abs() <= 2 * R_TOL * 2).any(-1)


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(128, 128, 0, 0), (256, 4096, 0, 0), (128, 640, 8, 8), (128, 384, 5, 3),
                                                  (384, 1024, 0, 0), (128, 16512, 0, 0), (128, 256, 1, 0)])
def test_codes(rows, cols, pad, offset, dtype, fmt, recipe):
    """The codes stand for y within half a step, the scales are the recipe's for y's amaxes; with binary32 data, whose y is
    kept unrounded, both are the bytes of the library's cast of y."""
    dt = DTYPES[dtype]
    x, res = matrix(rows, cols, dt, 5, pad, offset, 3.0), matrix(rows, cols, dt, 6, 0, 0, 2.0)
    x[3] = 0
    res[3] = 0                    # an all-zero row
    x[5, :32] *= 1e-3
    w = _weight(cols, torch.float32, 7)
    scale = torch.full((1,), FMAX[int(fmt)] / 3.0, device="cuda") if recipe == R.TENSOR else None
    amax = torch.full((1,), 9e9, device="cuda") if recipe == R.TENSOR else None
    y, h, rstd, q, s = fq.rms_norm(x, w, res, EPS, recipe=recipe, fmt=fmt, scale=scale, amax_out=amax)
    only = fq.rms_norm(x, w, res, EPS, recipe=recipe, fmt=fmt, scale=scale, amax_out=amax, keep_y=False, stats=False)
    assert only[0] is None and only[2] is None and torch.equal(only[3], q) and torch.equal(only[4], s) and torch.equal(only[1], h)
    _, _, y64 = _exact(x, res, w)
    if dtype == "fp32":
        qc, sc, _, _ = fq.cast_transpose(y, recipe, fmt, scale, col=False)
        assert torch.equal(q, qc)
        if recipe != R.TENSOR:
            assert torch.equal(s.view(torch.uint8), sc.view(torch.uint8))
    got = values(q, recipe, fmt, s)
    if recipe == R.TENSOR:
        assert_within(amax, y64.abs().max().reshape(1), R_TOL * y64.abs().max().reshape(1), "amax")
        assert torch.equal(s, 1 / scale)
        mult = s.double().expand(rows, cols)
    elif recipe == R.BLOCK_1x128:
        a = y64.view(rows, -1, 128).abs().amax(2)
        want = torch.where(a > 0, a / FMAX[int(fmt)], 1.0)
        assert_within(s, want, (R_TOL + 3 * U) * want, "multipliers")
        mult = s.double().repeat_interleave(128, 1)
    else:
        floor = recipe in (R.MX_1x32_FLOOR, R.MX_1x32_FLOOR_TILED)
        a = y64.view(rows, -1, 32).abs().amax(2)
        p = e8m0_values(s, rows, cols, recipe in (R.MX_1x32_TILED, R.MX_1x32_FLOOR_TILED))
        top = 8 if fmt == F.E4M3 else 15
        e = torch.floor(torch.log2(a.clamp(min=1e-300))) - top
        if not floor:
            e = e + (a / torch.exp2(e + top) > 1.75)
        want = torch.where(a > 0, torch.exp2(e), 1.0)
        assert bool(((p == want) | _near_border(a, fmt, floor)).all())
        mult = p.repeat_interleave(32, 1)
    # the nearest code is at most half a step away: 2^-4 (E4M3) or 2^-3 (E5M2) of the value, or half the smallest code; what
    # saturates (the floor rule, a per-tensor scale of the past) has its own value
    half, least = ((2.0 ** -4, 2.0 ** -10) if fmt == F.E4M3 else (2.0 ** -3, 2.0 ** -17))
    ref = y64.clamp(-FMAX[int(fmt)] * mult, FMAX[int(fmt)] * mult)
    assert_within(got, ref, y64.abs() * (half + 2 * R_TOL) + least * mult * (1 + 1e-6), "codes")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("recipe,cols", [(R.TENSOR, 1003), (R.BLOCK_1x128, 1003), (R.BLOCK_1x128, 70), (R.MX_1x32, 1056), (R.MX_1x32, 32),
                                         (R.TENSOR, 17), (R.BLOCK_1x128, 20011)])
def test_codes_of_odd_widths(recipe, cols, dtype):
    rows, dt, fmt = 37, DTYPES[dtype], F.E4M3
    x, w = matrix(rows, cols, dt, 8, 3, 1), _weight(cols, torch.float32, 9)
    scale = torch.full((1,), 100.0, device="cuda") if recipe == R.TENSOR else None
    y, h, rstd, q, s = fq.rms_norm(x, w, None, EPS, recipe=recipe, fmt=fmt, scale=scale)
    assert h is None and q.shape == (rows, cols)
    _, _, y64 = _exact(x, None, w)
    got = values(q, recipe, fmt, s)
    mult = got.new_ones(rows, cols) * (s.double() if recipe == R.TENSOR else 1)
    if recipe == R.BLOCK_1x128:
        assert s.shape == (rows, (cols + 127) // 128)
        a = torch.stack([p.abs().amax(1) for p in y64.split(128, 1)], 1)
        assert_within(s, a / 448, (R_TOL + 3 * U) * a / 448, "multipliers")
        mult = s.double().repeat_interleave(128, 1)[:, :cols]
    elif recipe == R.MX_1x32:
        mult = e8m0_values(s, rows, cols, False).repeat_interleave(32, 1)
    ref = y64.clamp(-448 * mult, 448 * mult)
    assert_within(got, ref, y64.abs() * (2.0 ** -4 + 2 * R_TOL) + 2.0 ** -10 * mult * (1 + 1e-6), "codes")


@pytest.mark.parametrize("recipe", [R.BLOCK_1x128, R.MX_1x32_TILED])
def test_codes_feed_the_product(recipe):
    """The 8-bit output is an operand of the FP8 product as it is."""
    rows, cols, n = 256, 512, 256
    x, w = matrix(rows, cols, torch.bfloat16, 10), _weight(cols, torch.float32, 11)
    rb = R.BLOCK_128x128 if recipe == R.BLOCK_1x128 else recipe
    wt = torch.randn((n, cols), generator=gen(12), device="cuda").bfloat16()
    qw, sw, _, _ = fq.cast_transpose(wt, rb, F.E4M3, col=False)
    _, _, _, q, s = fq.rms_norm(x, w, None, EPS, recipe=recipe, keep_y=False)
    c = fq.scaled_gemm(q, F.E4M3, recipe, s, qw, F.E4M3, rb, sw, fq.OutDtype.FP32).double()
    a = values(q, recipe, F.E4M3, s)
    if rb == R.BLOCK_128x128:
        b = qw.view(torch.float8_e4m3fn).double() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    else:
        b = values(qw, rb, F.E4M3, sw)
    assert_within(c, a @ b.t(), 2.0 ** -23 * (cols + 64) * (a.abs() @ b.abs().t()), "product")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("rows,cols,pad,offset", CASES)
def test_backward(rows, cols, pad, offset, stream, dtype):
    dt = DTYPES[dtype]
    h = matrix(rows, cols, dt, 21, pad, offset, 3.0)
    dy = matrix(rows, cols, dt, 22, pad // 2, offset, 1e-2)
    dh = matrix(rows, cols, dt, 23, pad, 0, 1e-2) if stream else None
    w = _weight(cols, torch.float32 if rows % 2 else torch.bfloat16, 24) if cols != 1024 else None
    rstd = (1 / (h.float().square().mean(1) + EPS).sqrt())
    dx, dw = fq.rms_norm_backward(dy, h, rstd, w, dh=dh)
    r, y = rstd.double()[:, None], dy.double()
    xh, g = h.double() * r, y * (1.0 if w is None else w.double())
    c = (g * xh).mean(1, keepdim=True)
    ref = r * (g - xh * c) + (0.0 if dh is None else dh.double())
    # c's sum as the forward pass's (55 U of the absolute terms' mean); a handful of products
    ctol = (R_TOL + 6 * U) * (g * xh).abs().mean(1, keepdim=True)
    tol = r * (4 * U * g.abs() + xh.abs() * (ctol + 6 * U * c.abs())) + 2 * U * ref.abs()
    assert_within(dx, ref, out_tol(ref, tol, dt), "dx")
    terms = y * xh
    dtype_w = torch.float32 if w is None else w.dtype
    tol = (rows + 48) * U * terms.abs().sum(0) + 2 * U * terms.abs().sum(0)
    assert_within(dw, terms.sum(0), out_tol(terms.sum(0), tol, dtype_w), "dweight")
    assert dw.dtype == dtype_w
    alone, none = fq.rms_norm_backward(dy, h, rstd, w, dh=dh, param_grads=False)
    assert none is None and torch.equal(alone, dx)


def test_backward_against_differences():
    """<dx, v> and <dweight, u> against central differences of the 64-bit forward pass."""
    rows, cols = 24, 200
    x, res, w = matrix(rows, cols, torch.float32, 31), matrix(rows, cols, torch.float32, 32), _weight(cols, torch.float32, 33)
    dy, dh = matrix(rows, cols, torch.float32, 34), matrix(rows, cols, torch.float32, 35)
    _, h, rstd, _, _ = fq.rms_norm(x, w, res, EPS)
    dx, dw = fq.rms_norm_backward(dy, h, rstd, w, dh=dh)

    def loss(h64, w64):
        r = 1 / (h64.square().mean(1, keepdim=True) + EPS).sqrt()
        return float(((h64 * r * w64) * dy.double()).sum() + (h64 * dh.double()).sum())

    h64, w64, step = h.double(), w.double(), 1e-4
    for seed in range(3):
        v = torch.randn((rows, cols), generator=gen(40 + seed), device="cuda").double()
        u = torch.randn(cols, generator=gen(50 + seed), device="cuda").double()
        for got, plus, minus in ((float((dx.double() * v).sum()), loss(h64 + step * v, w64), loss(h64 - step * v, w64)),
                                 (float((dw.double() * u).sum()), loss(h64, w64 + step * u), loss(h64, w64 - step * u))):
            # differences: step^2 of third derivatives and cancellation; binary32 gradients of 4800 terms
            assert abs(got - (plus - minus) / (2 * step)) <= 1e-5 * (1 + abs(got)) + 64 * U * 4800


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_special_rows(dtype):
    """NaN and infinities stay in their rows; a row of zeros gives zeros; squares past binary32 give r = 0."""
    dt = DTYPES[dtype]
    x = matrix(8, 512, dt, 61)
    x[1, 7] = float("nan")
    x[2, 500] = float("inf")
    x[3] = 0
    x[4] = 3e19
    y, _, rstd, q, s = fq.rms_norm(x, recipe=R.MX_1x32)
    clean = fq.rms_norm(x[[0, 3, 5, 6, 7]].contiguous(), recipe=R.MX_1x32)
    keep = [0, 3, 5, 6, 7]
    assert torch.equal(y[keep], clean[0]) and torch.equal(q[keep], clean[3]) and torch.equal(s[keep], clean[4])
    assert y[1].isnan().all() and y[2, 500].isnan() and (y[2, :500] == 0).all()
    assert (y[3] == 0).all() and (q[3] == 0).all() and (s[3] == 127).all() and (y[4] == 0).all() and rstd[4] == 0
    assert_status_ok()


def test_outputs_stay_inside():
    """Every output between guard regions, rows strided."""
    for rows, cols, dt in ((37, 1003, torch.bfloat16), (128, 384, torch.bfloat16), (5, 20011, torch.float32), (128, 640, torch.float32)):
        x, res, w = matrix(rows, cols, dt, 71), matrix(rows, cols, dt, 72), _weight(cols, torch.float32, 73)
        recipe = R.MX_1x32_TILED if rows == 128 else R.BLOCK_1x128
        shape, sdt = fq.scale_shape(recipe, rows, cols) if rows == 128 else ((rows, (cols + 127) // 128), torch.float32)
        h, y, q = Guarded((rows, cols), dt), Guarded((rows, cols), dt), Guarded((rows, cols), torch.uint8)
        s, r = Guarded(shape, sdt), Guarded((rows,), torch.float32)
        fq.fp8_rms_norm(x, res, w, EPS, h.t, y.t, r.t, recipe, F.E4M3, None, None, q.t, s.t)
        want = fq.rms_norm(x, w, res, EPS, recipe=recipe)
        for got, ref, what in ((y, want[0], "y"), (h, want[1], "h"), (r, want[2], "rstd"), (q, want[3], "q"), (s, want[4], "s")):
            got.check(what)
            assert torch.equal(got.t, ref), what
        dx, dw = Guarded((rows, cols), dt), Guarded((cols,), torch.float32)
        ws = Guarded((fq.fp8_rms_norm_workspace(rows, cols),), torch.uint8)
        fq.fp8_rms_norm_backward(res, x, r.t, None, w, dx.t, dw.t, ws.t)
        for got, what in ((dx, "dx"), (dw, "dweight"), (ws, "workspace")):
            got.check(what)
        want = fq.rms_norm_backward(res, x, r.t, w)
        assert torch.equal(dx.t, want[0]) and torch.equal(dw.t, want[1])


def test_empty():
    z = torch.empty((0, 64), device="cuda")
    amax = torch.full((1,), 5.0, device="cuda")
    one = torch.ones(1, device="cuda")
    y, h, rstd, q, s = fq.rms_norm(z, recipe=R.TENSOR, scale=one, amax_out=amax)
    assert y.shape == (0, 64) and q.shape == (0, 64) and rstd.shape == (0,) and float(amax) == 0
    assert fq.rms_norm(torch.empty((5, 0), device="cuda"))[0].shape == (5, 0)
    dx, dw = fq.rms_norm_backward(z, z, torch.empty(0, device="cuda"), torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and dw.shape == (64,) and (dw == 0).all()


def test_graph_and_streams():
    """Captured and replayed on new data, with a call on another stream between."""
    rows, cols = 300, 1536
    x, res, w = matrix(rows, cols, torch.bfloat16, 81), matrix(rows, cols, torch.bfloat16, 82), _weight(cols, torch.float32, 83)
    dy = matrix(rows, cols, torch.bfloat16, 84)

    def step():
        amax = torch.empty(1, device="cuda")
        out = fq.rms_norm(x, w, res, EPS, recipe=R.TENSOR, scale=torch.full((1,), 50.0, device="cuda"), amax_out=amax)
        return (*out, amax, *fq.rms_norm_backward(dy, out[1], out[2], w, dh=dy))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    x.copy_(matrix(rows, cols, torch.bfloat16, 85))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y = fq.rms_norm(x, w, res, EPS, stream=other)[0]
    other.synchronize()
    assert torch.equal(y, want[0])


MORE_ROWS = [  # rows, cols, pad, offset: above and at the rows that one launch takes
    (152, 5849, 0, 0), (153, 5849, 1, 1), (76, 1003, 6, 5), (77, 1003, 6, 5), (77, 9, 0, 0), (153, 8, 0, 0), (160, 1, 0, 0),
    (152, 8192, 0, 0), (153, 8192, 8, 0), (170, 12288, 0, 0), (155, 16383, 0, 1), (160, 16384, 0, 0), (154, 16392, 0, 0), (152, 20480, 0, 0),
    (200, 250, 6, 0), (400, 4099, 0, 0), (1300, 130, 2, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("rows,cols,pad,offset", MORE_ROWS)
def test_backward_of_more_rows(rows, cols, pad, offset, stream, dtype):
    test_backward(rows, cols, pad, offset, stream, dtype)


def test_backward_stays_inside_of_more_rows():
    for rows, cols, dt in ((170, 1003, torch.bfloat16), (160, 640, torch.float32), (153, 20011, torch.float32), (152, 130, torch.bfloat16)):
        dy, h, dh = (matrix(rows, cols, dt, 90 + i) for i in range(3))
        w = _weight(cols, torch.float32, 93)
        rstd = torch.rand(rows, generator=gen(94), device="cuda")
        dx, dw = Guarded((rows, cols), dt), Guarded((cols,), torch.float32)
        ws = Guarded((fq.fp8_rms_norm_workspace(rows, cols),), torch.uint8)
        fq.fp8_rms_norm_backward(dy, h, rstd, dh, w, dx.t, dw.t, ws.t)
        for got, what in ((dx, "dx"), (dw, "dweight"), (ws, "workspace")):
            got.check(what)
        want = fq.rms_norm_backward(dy, h, rstd, w, dh=dh)
        assert torch.equal(dx.t, want[0]) and torch.equal(dw.t, want[1])


@pytest.mark.parametrize("rows,cols", [(170, 96), (160, 99)])
def test_backward_of_more_rows_against_differences(rows, cols):
    x, w = matrix(rows, cols, torch.float32, 101), _weight(cols, torch.float32, 102)
    dy = matrix(rows, cols, torch.float32, 103)
    _, _, rstd, _, _ = fq.rms_norm(x, w, None, EPS)
    dx, dw = fq.rms_norm_backward(dy, x, rstd, w)

    def loss(h64, w64):
        return float((h64 / (h64.square().mean(1, keepdim=True) + EPS).sqrt() * w64 * dy.double()).sum())

    h64, w64, step = x.double(), w.double(), 1e-4
    v = torch.randn((rows, cols), generator=gen(104), device="cuda").double()
    u = torch.randn(cols, generator=gen(105), device="cuda").double()
    for got, plus, minus in ((float((dx.double() * v).sum()), loss(h64 + step * v, w64), loss(h64 - step * v, w64)),
                             (float((dw.double() * u).sum()), loss(h64, w64 + step * u), loss(h64, w64 - step * u))):
        assert abs(got - (plus - minus) / (2 * step)) <= 1e-5 * (1 + abs(got)) + 64 * U * rows * cols
