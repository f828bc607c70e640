"""SiLU and GELU tanh of bf16 data far below zero, where the sigmoid is small and then subnormal: no value
that the output's type holds is lost.

Tolerances, u = 2^-24: the sigmoid by an exponential of relative error (|z| + 8) u and a division and a
product of 6 u; GELU's tanh form rounds z to 6 u |z|.  f' = s + f (1 - s) z' adds 6 u of its terms.  One
rounding to bf16, whose subnormals are 2^-133 apart, and the smallest binary32 subnormal times what it is
multiplied by."""
import math

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import assert_status_ok, require_gpu
from row_util import BF16, U, assert_within

pytestmark = pytest.mark.gpu
A = fq.Activation


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("kind", [A.SILU, A.GELU_TANH])
@pytest.mark.parametrize("cols", [256, 101])          # 16-byte accesses, words
def test_small_sigmoids(kind, cols):
    low = -112.0 if kind == A.SILU else -11.5
    x = torch.linspace(low, low / 4, 10 * cols, device="cuda").to(torch.bfloat16).view(10, cols)
    y = fq.gated_act(x, None, kind)[0]
    da = fq.gated_act_backward(torch.ones_like(x), kind, a=x)[0]
    dga, dgb = fq.gated_act_backward(torch.full_like(x, 8.0), kind, a=x, b=torch.full_like(x, 4.0))
    assert_status_ok()
    xd = x.double()
    k = 2 * math.sqrt(2 / math.pi)
    z, dz, ez = (xd, torch.ones_like(xd), 1.0) if kind == A.SILU else (
        k * (xd + 0.044715 * xd ** 3), k * (1 + 3 * 0.044715 * xd * xd), 7.0)
    t = torch.exp(z)
    s, sc = t / (1 + t), 1 / (1 + t)
    f, df = xd * s, s + xd * s * sc * dz
    rel = (ez * z.abs() + 14) * U
    t_f, t_df = rel * f.abs(), (rel + 6 * U) * (s + (f * dz).abs())
    small = 2.0 ** -149 * (1 + xd.abs()) * (1 + dz.abs())
    for got, ref, tol, m, what in ((y, f, t_f, 1.0, "f"), (da, df, t_df, 1.0, "f'"), (dga, 32 * df, 32 * t_df, 32.0, "dy b f'"),
                                   (dgb, 8 * f, 8 * t_f, 8.0, "dy f")):
        assert_within(got, ref, tol + BF16 * (ref.abs() + tol) + 2.0 ** -133 + m * small, what)
