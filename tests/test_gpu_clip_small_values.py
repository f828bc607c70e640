"""The gradients' norm of small values: as near to the 64-bit sum, and as fast, as of ordinary ones."""
import math

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import require_gpu
from row_util import U, gen

pytestmark = pytest.mark.gpu

# A thread's 16 or 32 squares in two chains of at most 16 roundings, one addition, and binary64 beyond: 17 U of the sum.  Its root
# halves that; the sum rounded to binary32 and the root add U / 2 and U.
NORM_TOL = 10 * U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("exponent", [0, -8, -24, -28, -30, -32, -40, -50, -54, -55, -56, -57, -58, -59, -60, -64, -74, -90, -120])
def test_norm(exponent, dtype):
    """Around every magnitude at which the sums change their precision: 2^-30 squared is 2^-60, 2^-55 squared 2^-110."""
    g = [(torch.randn(n, generator=gen(n), device="cuda") * 2.0 ** exponent).to(dtype) for n in (100003, 64, 5)]
    ref = math.sqrt(math.fsum(float(x.double().square().sum()) for x in g))
    assert abs(float(fq.grad_norm(g)) - ref) <= NORM_TOL * ref
    by = min(1.0, 1e-30 / (ref + 1e-6))
    outs = [torch.empty_like(x) for x in g]
    assert abs(float(fq.clip_grad_norm(g, 1e-30, out=outs)) - ref) <= NORM_TOL * ref
    half = torch.finfo(dtype).eps / 2
    for x, o in zip(g, outs):
        want = x.double() * by
        assert bool(((o.double() - want).abs() <= want.abs() * (NORM_TOL + 4 * U + half) + 2.0 ** -133).all())


def test_mixed_magnitudes():
    """Lanes of tiny values beside lanes of large ones, zeros of either sign, a lone subnormal."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(1 << 16, generator=gen(1), device="cuda")
        e = torch.randint(-70, 10, (1 << 16,), generator=gen(2), device="cuda").float()
        g = (x * torch.exp2(e)).to(dtype)
        g[::7] = 0.0
        g[3::7] = -0.0
        for part in (g, g[:4096] * 2.0 ** -50, g[5:69] * 0.0 + 2.0 ** -130):
            part = part.to(dtype)
            ref = math.sqrt(float(part.double().square().sum()))
            assert abs(float(fq.grad_norm([part])) - ref) <= NORM_TOL * ref + 2.0 ** -150


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_gradients_take_no_longer(dtype):
    """Bound by memory: 200 MB of gradients near 1e-11 (a loss averaged over many tokens, a rarely routed expert) are read as fast
    as of 1e-3.  Sums in binary64 throughout would take several times as long; half as long again is neither."""
    n = 200_000_000 // dtype.itemsize
    x = torch.randn(n, generator=gen(3), device="cuda")
    grads = [(x * sigma).to(dtype) for sigma in (1e-3, 1e-11)]
    del x
    least = [math.inf, math.inf]
    for _ in range(12):
        for i, g in enumerate(grads):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            fq.grad_norm([g])
            b.record()
            torch.cuda.synchronize()
            least[i] = min(least[i], a.elapsed_time(b))
    assert least[1] <= 1.5 * least[0], least
