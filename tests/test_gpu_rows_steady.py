"""The row operators at sizes where every group of warps works on many rows: stages refilled, buffers
in turn, the next item fetched ahead, several sweeps of the largest grid.  The checks and their
tolerances are those of the operators' own tests; the numbers of rows follow from the GPU's SMs."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
import test_gpu_act as act
import test_gpu_moe as moe
import test_gpu_norm as norm
from gpu_util import F, assert_status_ok, require_gpu
from row_util import DTYPES, F8, FMAX, assert_within, code_values, matrix, out_tol

pytestmark = pytest.mark.gpu
A = fq.Activation
TURNS = 9        # rows of a group: more than twice the stages in flight (4 at most), and one


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def norm_rows(cols):
    """Rows that give every group of every block TURNS of them: a block an SM, as many groups as 32 warps can be."""
    values = 8 if cols <= 256 else 16 if cols <= 512 else 32
    warps = -(-cols // (32 * values))
    most = 32 if values == 8 else 24 if values == 16 else 24   # warps of a block
    return sms() * max(1, most // warps) * TURNS + 5


# a warp a row (8, 16 and 32 values a lane), several, widths of 5, 7 and 8 warps, the widest; odd and even, aligned and not
WIDTHS = [96, 128, 250, 256, 400, 512, 1000, 1024, 1003, 2560, 4096, 4099, 5120, 5121, 7168, 8192, 8200, 12288, 12301, 16381, 16384]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_forward(cols, dtype):
    norm.test_forward(norm_rows(cols), cols, dtype)


@pytest.mark.parametrize("cols", [128, 250, 512, 1003, 4096, 4099, 5120, 12301, 16384])
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_codes(cols, fmt, dtype):
    rows = norm_rows(cols)
    x = matrix(rows, cols, DTYPES[dtype], 1100 + cols)
    y, mean, rstd, q, s = fq.layer_norm(x, checkpoint=fmt)
    assert_status_ok()
    if dtype == "fp32":     # y is xh itself: the codes and multipliers are the recipe's, bit for bit
        wide = torch.zeros((rows, (cols + 127) // 128 * 128), device="cuda")
        wide[:, :cols] = y
        amax = wide.view(rows, -1, 128).abs().amax(2)
        scale = torch.where(amax > 0, torch.full_like(amax, FMAX[int(fmt)]) / amax, 1.0)
        assert torch.equal(s, torch.ones_like(scale) / scale)
        v = (wide.view(rows, -1, 128) * scale[..., None]).clamp(-FMAX[int(fmt)], FMAX[int(fmt)]).view(rows, -1)[:, :cols]
        assert torch.equal(q, v.to(F8[int(fmt)]).view(torch.uint8))
    _, _, xh, _, _, _, t_xh, _ = norm.reference(x, None, None, 1e-5)
    step, small = (2.0 ** -4, 2.0 ** -10) if fmt == F.E4M3 else (2.0 ** -3, 2.0 ** -17)
    mult = s.double().repeat_interleave(128, 1)[:, :cols]
    assert_within(code_values(q, s, fmt), xh, torch.maximum((xh.abs() + t_xh) * step, mult * small) + t_xh + 4 * norm.U * xh.abs(),
                  "values of the codes")


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("source", ["x", "e4m3", "e5m2"])
def test_norm_backward(cols, dtype, source):
    norm.test_backward(norm_rows(cols), cols, dtype, source)


@pytest.mark.parametrize("cols", [250, 1024, 4099, 5120])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 1)])
def test_norm_strides(cols, pad, offset):
    rows, dt = norm_rows(cols), torch.bfloat16
    x, y, dy, dx = (matrix(rows, cols, dt, 1200 + i, pad, offset) for i in range(4))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    w, b = norm.params(cols, torch.float32, 15)
    fq.fp8_layer_norm(x, w, b, 1e-5, y, mean, rstd, F.E4M3, None, None)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(fq.fp8_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    fq.fp8_layer_norm_backward(dy, x, mean, rstd, F.E4M3, None, None, w, dx, dw, db, ws)
    assert_status_ok()
    _, _, _, y_ref, _, _, _, t_y = norm.reference(x, w, b, 1e-5)
    assert_within(y, y_ref, out_tol(y_ref, t_y, dt), "y")
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    norm.check_backward((dx, dw, db), norm.backward_reference(dy, xh, rstd, w), dt, torch.float32)


def act_rows(cols, dtype):
    """Rows whose pieces are two and a half sweeps of the largest grid, 32 blocks of 8 warps an SM."""
    pieces = -(-cols // (512 if dtype == "bf16" else 256))
    return sms() * 32 * 8 * 5 // 2 // pieces + 3


@pytest.mark.parametrize("cols", [256, 1501, 1504, 9001])
@pytest.mark.parametrize("kind,gated", [(A.SILU, True), (A.GELU, False), (A.GELU_TANH, True)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_act(cols, kind, gated, dtype):
    rows = act_rows(cols, dtype)
    act.test_forward(rows, cols, kind, gated, dtype)
    act.test_backward(rows, cols, kind, gated, dtype, "x")
    act.test_backward(rows, cols, kind, gated, dtype, "e4m3")


@pytest.mark.parametrize("cols", [256, 1501, 1504])
@pytest.mark.parametrize("dtype", DTYPES)
def test_act_codes(cols, dtype):
    rows, fmt = act_rows(cols, dtype), F.E4M3
    a, b = matrix(rows, cols, DTYPES[dtype], 1300), matrix(rows, cols, DTYPES[dtype], 1301, sigma=30.0)
    _, qa, sa, qb, sb = fq.gated_act(a, b, A.SILU, checkpoint=fmt)
    assert_status_ok()
    for x, q, s in ((a, qa, sa), (b, qb, sb)):
        wide = torch.zeros((rows, (cols + 127) // 128 * 128), device="cuda")
        wide[:, :cols] = x
        amax = wide.view(rows, -1, 128).abs().amax(2)
        scale = torch.where(amax > 0, torch.full_like(amax, FMAX[int(fmt)]) / amax, 1.0)
        assert torch.equal(s, torch.ones_like(scale) / scale)
        v = (wide.view(rows, -1, 128) * scale[..., None]).clamp(-FMAX[int(fmt)], FMAX[int(fmt)]).view(rows, -1)[:, :cols]
        assert torch.equal(q, v.to(F8[int(fmt)]).view(torch.uint8))


# tokens for several sweeps of dispatch's grid (16 blocks an SM, 8 warps' worth of tokens a block) and of the others'
# (8); one and several warps a token, rows that a block goes over twice; then more choices than a warp has lanes
MOE = [(60000, 2, 8, 264, 128), (60000, 1, 64, 250, 1), (16000, 3, 8, 1500, 16), (16000, 3, 8, 1501, 16), (8000, 2, 16, 5003, 128),
       (8000, 4, 16, 4096, 128), (6000, 8, 64, 2048, 128), (3000, 2, 4, 12296, 1), (3000, 40, 64, 1000, 16), (2500, 40, 48, 1001, 1),
       (700, 33, 64, 4096, 8), (9, 70, 128, 520, 1), (300, 64, 64, 5003, 128)]


@pytest.mark.parametrize("tokens,k,n_experts,cols,align", MOE)
@pytest.mark.parametrize("dtype", DTYPES)
def test_dispatch_and_combine(tokens, k, n_experts, cols, align, dtype):
    moe.test_dispatch_and_combine(tokens, k, n_experts, cols, align, dtype)


@pytest.mark.parametrize("tokens,k,n_experts,cols,align", MOE)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_backward(tokens, k, n_experts, cols, align, dtype):
    moe.test_combine_backward(tokens, k, n_experts, cols, align, dtype)


def test_the_same_bits_every_time():
    for cols in (1003, 4096, 5120):
        rows = norm_rows(cols)
        x, dy = matrix(rows, cols, torch.bfloat16, 1400), matrix(rows, cols, torch.bfloat16, 1401)
        first = None
        for _ in range(3):
            y, mean, rstd, q, s = fq.layer_norm(x, checkpoint=F.E4M3)
            out = [y, mean, rstd, q, s, *fq.layer_norm_backward(dy, rstd, x=x, mean=mean), *fq.layer_norm_backward(dy, rstd, q=q, s=s)]
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, out))
            first = out
    assert_status_ok()
