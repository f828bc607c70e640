"""Layer norm, forward and backward, against the formulas in 64 bits.

Tolerances, with u = 2^-24 and K = ceil(cols / 32) + 16 (the longest chain of additions of a
kernel that spreads a row over a warp or more, plus the operations around the sums):
  the mean is off by at most e_m = K u mean|x|; the differences x - m by e_m + u |x - m|; so r by
  r (K u + r e_m) and xh by |xh| (K u + r e_m + 2 u) + r e_m, and y = xh w + b by |w| times that
  and u (|xh w| + |b|).
  dx = r (g - c1 - xh c2) with xh given to 2 u: off by K u r (|g| + mean|g| + 2 |xh| mean|g xh|).
  dw, db: (rows + 4) u times the sum of the terms' magnitudes, for any order of summation.
One rounding to the output's type is added (row_util.out_tol)."""
import numpy as np
import pytest
import torch

import oracle
import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import F, Guarded, assert_bytes_equal, assert_status_ok, f32bits, host, require_gpu
from row_util import DTYPES, U, assert_within, code_values, codes_of, matrix, out_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


SHAPES = [(1, 1), (5, 7), (3, 64), (2, 127), (257, 128), (4, 129), (33, 1000), (1, 4096), (70, 4096), (7, 5003),
          (5, 8192), (3, 12288), (2, 16392), (2, 33024), (2, 70001)]


def params(cols, wdt, seed):
    w = matrix(1, cols, wdt, seed, sigma=0.3)[0] + 1
    return w.contiguous(), matrix(1, cols, wdt, seed + 1, sigma=0.3)[0].contiguous()


def chain(cols):
    return (cols + 31) // 32 + 16


def reference(x, w, b, eps):
    """mean, rstd, xh, y and the tolerances of mean, rstd, xh, y."""
    x = x.double()
    cols = x.shape[1]
    m = x.mean(1, keepdim=True)
    r = 1 / ((x - m).square().mean(1, keepdim=True) + eps).sqrt()
    xh = (x - m) * r
    w = torch.ones(cols, dtype=torch.float64, device="cuda") if w is None else w.double()
    b = torch.zeros(cols, dtype=torch.float64, device="cuda") if b is None else b.double()
    y = xh * w + b
    ku = chain(cols) * U
    e_m = ku * x.abs().mean(1, keepdim=True)
    rel = ku + r * e_m
    e_xh = xh.abs() * (rel + 2 * U) + r * e_m
    return m, r, xh, y, e_m, r * rel, e_xh, e_xh * w.abs() + U * ((xh * w).abs() + b.abs())


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_forward(rows, cols, dtype):
    dt = DTYPES[dtype]
    x = matrix(rows, cols, dt, 100 + cols) + 0.5
    w, b = params(cols, torch.float32, 7)
    y, mean, rstd, _, _ = fq.layer_norm(x, w, b, 1e-5)
    assert_status_ok()
    m, r, _, y_ref, t_m, t_r, _, t_y = reference(x, w, b, 1e-5)
    assert y.dtype == dt
    assert_within(mean, m[:, 0], t_m[:, 0] + U * m[:, 0].abs(), "mean")
    assert_within(rstd, r[:, 0], t_r[:, 0] + U * r[:, 0], "rstd")
    assert_within(y, y_ref, out_tol(y_ref, t_y, dt), "y")


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (16, 8), (1, 5)])
@pytest.mark.parametrize("cols", [256, 1000, 4096])
@pytest.mark.parametrize("dtype", DTYPES)
def test_forward_strides_and_alignments(pad, offset, cols, dtype):
    dt = DTYPES[dtype]
    x = matrix(37, cols, dt, 200, pad, offset)
    out = matrix(37, cols, dt, 201, pad, offset)
    w, b = params(cols, torch.bfloat16, 8)
    fq.fp8_layer_norm(x, w, b, 1e-5, out, None, None, F.E4M3, None, None)
    assert_status_ok()
    _, _, _, y_ref, _, _, _, t_y = reference(x, w, b, 1e-5)
    assert_within(out, y_ref, out_tol(y_ref, t_y, dt), "y")


@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 7), (9, 127), (33, 128), (6, 1000), (40, 4096), (3, 5003), (5, 12288),
                                       (2, 33024)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_eight_bit_rows_are_the_blockwise_copy(rows, cols, dtype, fmt):
    # without weight and bias a binary32 y is xh itself; the codes and multipliers are the
    # 1x128 recipe's of those values, bit for bit (the ragged last block as if padded with 0)
    x = matrix(rows, cols, torch.float32, 300 + cols)
    x = x if dtype == "fp32" else x.to(torch.bfloat16)
    _, _, _, q, s = fq.layer_norm(x, checkpoint=fmt)
    y32, _, _, q32, s32 = fq.layer_norm(x.float(), checkpoint=fmt)
    assert_status_ok()
    wide = np.zeros((rows, (cols + 127) // 128 * 128), np.float32)
    wide[:, :cols] = host(y32)
    q_ref, s_ref = oracle.quantize_rowwise_f32(wide, oracle.KIND_1x128, int(fmt))
    assert_bytes_equal(host(q32), q_ref[:, :cols], "codes")
    assert_bytes_equal(f32bits(host(s32)), f32bits(s_ref), "multipliers")
    # a bf16 input holds the same values: the same codes up to the order of the row sums
    _, _, xh, _, _, _, t_xh, _ = reference(x, None, None, 1e-5)
    step, small = (2.0 ** -4, 2.0 ** -10) if fmt == F.E4M3 else (2.0 ** -3, 2.0 ** -17)
    mult = s.double().repeat_interleave(128, 1)[:, :cols]
    assert_within(code_values(q, s, fmt), xh, torch.maximum((xh.abs() + t_xh) * step, mult * small) + t_xh + 4 * U * xh.abs(),
                  "values of the codes")


def test_constant_and_non_finite_rows():
    x = torch.randn((6, 512), device="cuda")
    x[0] = 3.0                                   # no variance: xh = 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = torch.finfo(torch.bfloat16).min * 2.0 ** -70   # equal large values: no variance either
    w, b = params(512, torch.float32, 9)
    y, _, _, q, s = fq.layer_norm(x, w, b, 1e-5, checkpoint=F.E4M3)
    assert_status_ok()
    assert torch.equal(y[0], b) and torch.equal(q[0], torch.zeros_like(q[0])) and bool((s[0] == 1).all())
    assert torch.equal(y[3], b)
    assert bool(y[1].isnan().all()) and bool(y[2].isnan().all())
    _, _, _, y_ref, _, _, _, t_y = reference(x[4:], w, b, 1e-5)
    assert_within(y[4:], y_ref, out_tol(y_ref, t_y, torch.float32), "rows beside NaN")


def backward_reference(dy, xh, r, w):
    dy, r = dy.double(), r.double()[:, None]
    rows, cols = dy.shape
    g = dy if w is None else dy * w.double()
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    ku = chain(cols) * U
    t_dx = ku * r * (g.abs() + g.abs().mean(1, keepdim=True) + 2 * xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    ru = (rows + 4) * U
    return (r * (g - c1 - xh * c2), (dy * xh).sum(0), dy.sum(0), t_dx, ru * (dy * xh).abs().sum(0), ru * dy.abs().sum(0))


def check_backward(got, ref, dt, wdt):
    dx, dw, db, t_dx, t_dw, t_db = ref
    assert got[0].dtype == dt and got[1].dtype == wdt and got[2].dtype == wdt
    assert_within(got[0], dx, out_tol(dx, t_dx, dt), "dx")
    assert_within(got[1], dw, out_tol(dw, t_dw, wdt), "dweight")
    assert_within(got[2], db, out_tol(db, t_db, wdt), "dbias")


@pytest.mark.parametrize("rows,cols", SHAPES + [(1500, 640), (700, 4096), (400, 96)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("source", ["x", "e4m3", "e5m2"])
def test_backward(rows, cols, dtype, source):
    dt, wdt = DTYPES[dtype], torch.bfloat16 if cols % 2 else torch.float32
    dy = matrix(rows, cols, dt, 400 + cols)
    w, _ = params(cols, wdt, 10)
    if source == "x":
        x = matrix(rows, cols, dt, 401 + cols)
        mean = x.float().mean(1)
        rstd = 1 / (x.float().var(1, unbiased=False) + 1e-5).sqrt()
        xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
        got = fq.layer_norm_backward(dy, rstd, w, x=x, mean=mean)
    else:
        fmt = F.E4M3 if source == "e4m3" else F.E5M2
        q, s = codes_of(rows, cols, fmt, 402 + cols, pad=(16 - cols % 16) % 16)
        rstd = 0.5 + torch.rand(rows, device="cuda")
        xh = code_values(q, s, fmt)
        got = fq.layer_norm_backward(dy, rstd, w, q=q, s=s, fmt=fmt)
    assert_status_ok()
    check_backward(got, backward_reference(dy, xh, rstd, w), dt, wdt)


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (16, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_strides_and_alignments(pad, offset, dtype):
    dt, cols, rows = DTYPES[dtype], 1024, 45
    dy, x = matrix(rows, cols, dt, 500, pad, offset), matrix(rows, cols, dt, 501, pad, 0)
    dx = matrix(rows, cols, dt, 502, 0, offset)
    mean, rstd = torch.randn(rows, device="cuda"), 0.5 + torch.rand(rows, device="cuda")
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(fq.fp8_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    fq.fp8_layer_norm_backward(dy, x, mean, rstd, F.E4M3, None, None, None, dx, dw, db, ws)
    assert_status_ok()
    check_backward((dx, dw, db), backward_reference(dy, xh, rstd, None), dt, torch.float32)


def test_backward_without_parameter_gradients_and_of_no_rows():
    dy, x = matrix(20, 384, torch.bfloat16, 510), matrix(20, 384, torch.bfloat16, 511)
    mean, rstd = torch.zeros(20, device="cuda"), torch.ones(20, device="cuda")
    dx, dw, db = fq.layer_norm_backward(dy, rstd, x=x, mean=mean, param_grads=False)
    assert dw is None and db is None
    ref = backward_reference(dy, x.double(), rstd, None)
    assert_within(dx, ref[0], out_tol(ref[0], ref[3], torch.bfloat16), "dx")
    # one of the two alone
    for k in (1, 2):
        outs = [None, torch.empty(384, device="cuda") if k == 1 else None, torch.empty(384, device="cuda") if k == 2 else None]
        ws = torch.empty(fq.fp8_layer_norm_workspace(20, 384), dtype=torch.uint8, device="cuda")
        fq.fp8_layer_norm_backward(dy, x, mean, rstd, F.E4M3, None, None, None, dx, outs[1], outs[2], ws)
        assert_within(outs[k], ref[k], out_tol(ref[k], ref[k + 3], torch.float32), "one parameter gradient")
    none = torch.empty((0, 384), dtype=torch.bfloat16, device="cuda")
    dx, dw, db = fq.layer_norm_backward(none, rstd[:0], x=none, mean=mean[:0])
    assert_status_ok()
    assert dx.shape == (0, 384) and not bool(dw.any()) and not bool(db.any())
    assert fq.layer_norm(none)[0].shape == (0, 384)


def test_gradient_against_differences():
    # <grad, v> against the central difference of <dy, layer_norm(x + h v)> in 64 bits: the
    # difference's own error is O(h^2), 1e-8 relative here; binary32 gives about 1e-6
    x, w, b = matrix(11, 300, torch.float32, 520), *params(300, torch.float32, 11)
    dy, v = matrix(11, 300, torch.float32, 521), matrix(11, 300, torch.float32, 522)
    _, mean, rstd, _, _ = fq.layer_norm(x, w, b, 1e-5)
    dx, dw, db = fq.layer_norm_backward(dy, rstd, w, x=x, mean=mean)

    def loss(x, w, b):
        return (dy.double() * reference(x, w, b, 1e-5)[3]).sum()

    h = 1e-4
    vw = matrix(1, 300, torch.float32, 523)[0].double()
    x, w, b, v = x.double(), w.double(), b.double(), v.double()
    for name, grad, way, diff in (
            ("x", dx, v, loss(x + h * v, w, b) - loss(x - h * v, w, b)),
            ("weight", dw, vw, loss(x, w + h * vw, b) - loss(x, w - h * vw, b)),
            ("bias", db, vw, loss(x, w, b + h * vw) - loss(x, w, b - h * vw))):
        size = (grad.double() * way).abs().sum()
        assert abs((grad.double() * way).sum() - diff / (2 * h)) <= 2e-5 * size, name


def test_writes_stay_inside_and_repeat_bit_for_bit():
    for rows, cols in ((37, 1001), (65, 4096)):
        x, dy = matrix(rows, cols, torch.bfloat16, 530), matrix(rows, cols, torch.bfloat16, 531)
        first = None
        for _ in range(2):
            g = {n: Guarded(shape, dt) for n, shape, dt in (
                ("y", (rows, cols), torch.bfloat16), ("mean", (rows,), torch.float32), ("rstd", (rows,), torch.float32),
                ("q", (rows, cols), torch.uint8), ("s", (rows, (cols + 127) // 128), torch.float32),
                ("dx", (rows, cols), torch.bfloat16), ("dw", (cols,), torch.float32), ("db", (cols,), torch.float32),
                ("ws", (fq.fp8_layer_norm_workspace(rows, cols),), torch.uint8))}
            t = {n: v.t for n, v in g.items()}
            fq.fp8_layer_norm(x, None, None, 1e-5, t["y"], t["mean"], t["rstd"], F.E4M3, t["q"], t["s"])
            fq.fp8_layer_norm_backward(dy, None, None, t["rstd"], F.E4M3, t["q"], t["s"], None, t["dx"], t["dw"], t["db"],
                                       t["ws"])
            assert_status_ok()
            for n, v in g.items():
                v.check(n)
            outs = [host(t[n].view(torch.uint8)).copy() for n in ("y", "q", "s", "dx", "dw", "db")]
            if first is not None:
                for a, c in zip(first, outs):
                    assert np.array_equal(a, c)
            first = outs


def test_another_stream_and_a_graph():
    x, dy = matrix(64, 2048, torch.bfloat16, 540), matrix(64, 2048, torch.bfloat16, 541)
    w, b = params(2048, torch.float32, 12)
    y0, mean, rstd, q, s = fq.layer_norm(x, w, b, checkpoint=F.E4M3)
    ref = fq.layer_norm_backward(dy, rstd, w, q=q, s=s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        # work queued on the stream just before: the operator has to wait for it
        x2 = torch.zeros_like(x)
        for _ in range(20):
            x2.add_(x / 20 * 0)
        x2.add_(x)
        y1 = fq.layer_norm(x2, w, b)[0]
    side.synchronize()
    assert torch.equal(y0, y1)
    static = [torch.empty_like(t) for t in ref]
    ws = torch.empty(fq.fp8_layer_norm_workspace(64, 2048), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fp8_layer_norm_backward(dy, None, None, rstd, F.E4M3, q, s, w, *static, ws)
    for _ in range(2):
        for t in static:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(ref, static):
            assert torch.equal(a, c)


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_stream_owns_the_workspace(raw):
    # the call returns while its kernels wait behind other work of that stream; what it allocated for
    # itself must not be handed to the current stream meanwhile
    x, dy = matrix(64, 2048, torch.bfloat16, 542), matrix(64, 2048, torch.bfloat16, 543)
    w, b = params(2048, torch.float32, 13)
    _, mean, rstd, _, _ = fq.layer_norm(x, w, b)
    ref = fq.layer_norm_backward(dy, rstd, w, x=x, mean=mean)
    nbytes = fq.fp8_layer_norm_workspace(64, 2048)
    side = torch.cuda.Stream()
    big = torch.ones((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            out = big @ big
    got = fq.layer_norm_backward(dy, rstd, w, x=x, mean=mean, stream=side.cuda_stream if raw else side)
    junk = [torch.full((nbytes,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for a, c in zip(ref, got):
        assert torch.equal(a, c)
    del out, junk


def test_offsets_past_32_bits():
    ld = 1_200_000_000                            # the third row starts past 2^31 elements
    buf = torch.empty(2 * ld + 4096, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 4096), (ld, 1))
    x.copy_(matrix(3, 4096, torch.bfloat16, 550))
    y, mean, rstd, _, _ = fq.layer_norm(x)
    dense = x.contiguous()
    assert torch.equal(y, fq.layer_norm(dense)[0])
    dy = matrix(3, 4096, torch.bfloat16, 551)
    a, c = fq.layer_norm_backward(dy, rstd, x=x, mean=mean), fq.layer_norm_backward(dy, rstd, x=dense, mean=mean)
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    assert_status_ok()
