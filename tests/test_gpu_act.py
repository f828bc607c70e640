"""Gated and plain activations, forward and backward, against the formulas in 64 bits.

Tolerances, u = 2^-24.  The sigmoid s of an argument z, by an exponential of relative error
(|z| + 4) u (its argument is rounded after a product) and a division of 3 u, is off by
s (1 - s) (|z| + 6) u + 4 s u; GELU's tanh form rounds z itself to 5 u |z|.  The normal
distribution function P is held to 2^-22 absolute (4 half-steps of values near 1).
  f = x s: |x| times that and 2 u |f|;  f' = s + x s (1 - s) z': the error of s times
  (1 + |x z'|) and 8 u |x s (1 - s) z'|;  GELU's f' = P + x p(x): 2^-22 and (x^2 + 8) u |x p|.
The products with b and dy add 2 u, the output one rounding (row_util.out_tol)."""
import math

import numpy as np
import pytest
import torch

import oracle
import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import F, Guarded, assert_bytes_equal, assert_status_ok, bits16, f32bits, host, require_gpu
from row_util import BF16, DTYPES, TINY, U, assert_within, code_values, codes_of, matrix, out_tol

pytestmark = pytest.mark.gpu

A = fq.Activation
KINDS = [A.SILU, A.GELU, A.GELU_TANH]
SHAPES = [(1, 1), (5, 7), (3, 127), (65, 128), (4, 129), (33, 1000), (1, 11008), (9, 5003), (300, 256), (3, 49152)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def f_ref(kind, x):
    """f, f' and their tolerances."""
    if kind == A.GELU:
        cdf = 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
        pdf = torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        t = 2.0 ** -22
        return x * cdf, cdf + x * pdf, x.abs() * (t + 2 * U * cdf), t + (x * x + 8) * U * (x * pdf).abs()
    k = 2 * math.sqrt(2 / math.pi)
    z, dz, ez = (x, torch.ones_like(x), 1.0) if kind == A.SILU else (
        k * (x + 0.044715 * x ** 3), k * (1 + 3 * 0.044715 * x * x), 6.0)
    s = torch.sigmoid(z)
    sc = torch.sigmoid(-z)
    t_s = s * sc * (ez * z.abs() + 6) * U + 4 * s * U
    f, df = x * s, s + x * s * sc * dz
    return f, df, x.abs() * t_s + 2 * U * f.abs(), t_s * (1 + (x * dz).abs()) + 8 * U * (x * s * sc * dz).abs()


def forward_ref(kind, a, b):
    a = a.double()
    f, _, t, _ = f_ref(kind, a)
    if b is None:
        return f, t
    return f * b.double(), (t + 2 * U * f.abs()) * b.double().abs()


def backward_ref(kind, dy, a, b):
    f, df, tf, td = f_ref(kind, a)
    dy = dy.double()
    c = dy if b is None else dy * b
    return c * df, c.abs() * (td + 3 * U * df.abs()), dy * f, dy.abs() * (tf + 2 * U * f.abs())


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_forward(rows, cols, kind, gated, dtype):
    dt = DTYPES[dtype]
    h = matrix(rows, 2 * cols, dt, 600 + cols, sigma=3.0)
    a, b = h[:, :cols], h[:, cols:] if gated else None
    y = fq.gated_act(a, b, kind)[0]
    assert_status_ok()
    ref, tol = forward_ref(kind, a, b)
    assert y.dtype == dt
    assert_within(y, ref, out_tol(ref, tol, dt), "y")


@pytest.mark.parametrize("kind", KINDS)
def test_whole_range_of_arguments(kind):
    x = torch.cat([torch.linspace(-200, 200, 4001, device="cuda"), torch.tensor([0.0, 1e-30, -1e-30, 1e4, -1e4, 1e9, -1e9],
                                                                                   device="cuda")])[None]
    y = fq.gated_act(x, None, kind)[0]
    dx = fq.gated_act_backward(torch.ones_like(x), kind, a=x)[0]
    assert_status_ok()
    f, df, tf, td = f_ref(kind, x.double())
    assert_within(y, f, out_tol(f, tf + TINY * x.double().abs(), torch.float32), "f")
    assert_within(dx, df, out_tol(df, td + TINY * x.double().abs() ** 3, torch.float32), "f'")
    nan = torch.full((1, 8), float("nan"), device="cuda")
    assert bool(fq.gated_act(nan, None, kind)[0].isnan().all())
    assert bool(fq.gated_act_backward(torch.ones_like(nan), kind, a=nan)[0].isnan().all())


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (16, 8)])
@pytest.mark.parametrize("cols", [512, 1000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_alignments(pad, offset, cols, dtype):
    dt, rows = DTYPES[dtype], 29
    a, b, dy = (matrix(rows, cols, dt, 610 + i, pad, offset) for i in range(3))
    y, da, db = (matrix(rows, cols, dt, 620 + i, pad, offset) for i in range(3))
    fq.fp8_gated_act(a, b, A.SILU, y, F.E4M3, None, None, None, None)
    fq.fp8_gated_act_backward(dy, A.SILU, a, b, F.E4M3, None, None, None, None, da, db)
    assert_status_ok()
    ref, tol = forward_ref(A.SILU, a, b)
    assert_within(y, ref, out_tol(ref, tol, dt), "y")
    r = backward_ref(A.SILU, dy, a.double(), b.double())
    assert_within(da, r[0], out_tol(r[0], r[1], dt), "da")
    assert_within(db, r[2], out_tol(r[2], r[3], dt), "db")


@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 127), (33, 128), (6, 1000), (40, 4096), (3, 5003)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_eight_bit_inputs_are_the_blockwise_copy(rows, cols, dtype, fmt):
    dt = DTYPES[dtype]
    a, b = matrix(rows, cols, dt, 630), matrix(rows, cols, dt, 631, sigma=40.0)
    a[0, 0] = 0.0
    b[rows - 1] = 0.0                              # a row whose blocks are all zero
    if cols > 5:
        a[rows // 2, 3], a[rows // 2, 4], b[0, 5] = float("nan"), float("inf"), 3e38
    y, qa, sa, qb, sb = fq.gated_act(a, b, A.SILU, checkpoint=fmt)
    y0 = fq.gated_act(a, b, A.SILU)[0]
    assert_status_ok()
    assert_bytes_equal(host(y.contiguous().view(torch.uint8)), host(y0.view(torch.uint8)), "y with and without the copies")
    for name, x, q, s in (("a", a, qa, sa), ("b", b, qb, sb)):
        wide = torch.zeros((rows, (cols + 127) // 128 * 128), dtype=dt, device="cuda")
        wide[:, :cols] = x
        if dt == torch.bfloat16:
            q_ref, s_ref = oracle.quantize_rowwise(bits16(wide), oracle.KIND_1x128, int(fmt))
        else:
            q_ref, s_ref = oracle.quantize_rowwise_f32(host(wide), oracle.KIND_1x128, int(fmt))
        nan = host(x.isnan())
        assert_bytes_equal(np.where(nan, 0, host(q)), np.where(nan, 0, q_ref[:, :cols]), f"codes of {name}")
        assert bool(code_values(q, s, fmt)[x.isnan()].isnan().all())
        assert_bytes_equal(f32bits(host(s)), f32bits(s_ref), f"multipliers of {name}")
    if cols % 128 == 0:   # the dense copy is one that fp8_dequantize reads
        back = fq.dequantize(qb, fq.Recipe.BLOCK_1x128, fmt, sb)
        v = code_values(qb, sb, fmt)
        assert_within(back, v, BF16 * v.abs() + TINY, "fp8_dequantize of the copy")


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("source", ["x", "e4m3", "e5m2"])
def test_backward(rows, cols, kind, gated, dtype, source):
    dt = DTYPES[dtype]
    dy = matrix(rows, cols, dt, 640 + cols)
    if source == "x":
        a, b = matrix(rows, cols, dt, 641, sigma=2.0), matrix(rows, cols, dt, 642) if gated else None
        da, db = fq.gated_act_backward(dy, kind, a=a, b=b)
        a, b = a.double(), b.double() if gated else None
    else:
        fmt = F.E4M3 if source == "e4m3" else F.E5M2
        qa, sa = codes_of(rows, cols, fmt, 643, pad=(16 - cols % 16) % 16)
        qb, sb = codes_of(rows, cols, fmt, 644, pad=(16 - cols % 16) % 16) if gated else (None, None)
        da, db = fq.gated_act_backward(dy, kind, qa=qa, sa=sa, qb=qb, sb=sb, fmt=fmt)
        # the kernel's product of a code and its multiplier is rounded to binary32: its values
        # are the inputs of the formula
        a = code_values(qa, sa, fmt).float().double()
        b = code_values(qb, sb, fmt).float().double() if gated else None
    assert_status_ok()
    r = backward_ref(kind, dy, a, b)
    assert_within(da, r[0], out_tol(r[0], r[1], dt), "da")
    if gated:
        assert_within(db, r[2], out_tol(r[2], r[3], dt), "db")
    else:
        assert db is None


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_against_differences(kind):
    # central differences of the 64-bit forward, error O(h^2); binary32 gives about 1e-6
    a, b, dy = (matrix(7, 260, torch.float32, 650 + i) for i in range(3))
    va, vb = (matrix(7, 260, torch.float32, 660 + i).double() for i in range(2))
    da, db = fq.gated_act_backward(dy, kind, a=a, b=b)
    a, b, h = a.double(), b.double(), 1e-4

    def loss(a, b):
        return (dy.double() * f_ref(kind, a)[0] * b).sum()

    for grad, way, diff in ((da, va, loss(a + h * va, b) - loss(a - h * va, b)),
                            (db, vb, loss(a, b + h * vb) - loss(a, b - h * vb))):
        size = (grad.double() * way).abs().sum()
        assert abs((grad.double() * way).sum() - diff / (2 * h)) <= 2e-5 * size


def test_writes_stay_inside():
    for rows, cols in ((37, 1001), (65, 1024)):
        a, b, dy = (matrix(rows, cols, torch.bfloat16, 670 + i) for i in range(3))
        groups = (cols + 127) // 128
        g = {n: Guarded(shape, dt) for n, shape, dt in (
            ("y", (rows, cols), torch.bfloat16), ("qa", (rows, cols), torch.uint8), ("qb", (rows, cols), torch.uint8),
            ("sa", (rows, groups), torch.float32), ("sb", (rows, groups), torch.float32),
            ("da", (rows, cols), torch.bfloat16), ("db", (rows, cols), torch.bfloat16))}
        t = {n: v.t for n, v in g.items()}
        fq.fp8_gated_act(a, b, A.GELU, t["y"], F.E4M3, t["qa"], t["sa"], t["qb"], t["sb"])
        fq.fp8_gated_act_backward(dy, A.GELU, None, None, F.E4M3, t["qa"], t["sa"], t["qb"], t["sb"], t["da"], t["db"])
        assert_status_ok()
        for n, v in g.items():
            v.check(n)


def test_another_stream_and_no_rows():
    a, b = matrix(64, 2048, torch.bfloat16, 680), matrix(64, 2048, torch.bfloat16, 681)
    y0 = fq.gated_act(a, b)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a2 = torch.zeros_like(a)
        for _ in range(20):
            a2.add_(a * 0)
        a2.add_(a)
        y1 = fq.gated_act(a2, b)[0]
    side.synchronize()
    assert torch.equal(y0, y1)
    assert fq.gated_act(a[:0], b[:0], checkpoint=F.E4M3)[1].shape == (0, 2048)
    da, db = fq.gated_act_backward(a[:0], a=a[:0], b=b[:0])
    assert da.shape == db.shape == (0, 2048)
    assert_status_ok()


def test_offsets_past_32_bits():
    ld = 1_200_000_000
    buf = torch.empty(2 * ld + 4096, dtype=torch.bfloat16, device="cuda")
    a = buf.as_strided((3, 4096), (ld, 1))
    a.copy_(matrix(3, 4096, torch.bfloat16, 690))
    dy, dense = matrix(3, 4096, torch.bfloat16, 691), a.contiguous()
    assert torch.equal(fq.gated_act(a)[0], fq.gated_act(dense)[0])
    assert torch.equal(fq.gated_act_backward(dy, a=a)[0], fq.gated_act_backward(dy, a=dense)[0])
    assert_status_ok()
