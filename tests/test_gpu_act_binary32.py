"""The activations of binary32 data, to binary32's own accuracy everywhere: relative to the value, also
where it is small.

Tolerances, u = 2^-24: the accuracy asked for is that of a direct evaluation with CUDA's functions, by
the error bounds stated for them (expf 2 units in the last place, 4 u; normcdff 5, 10 u) and one
rounding an operation:
  s = 1 / (1 + t) or t / (1 + t) with t = exp(-|z|): 4 u for t, 5 u for 1 + t, 2 u for division and
  product: 12 u of s, and of 1 - s alike.  GELU's tanh form rounds z itself to 5 u |z| (6 u with the
  formula's constants), which moves s by s (1 - s) times that.
  f = x s: 13 u of f.  f' = s + f (1 - s) z': 12 u of s, 36 u of the product.
  GELU: P to 10 u; p(x), whose exponent is rounded to u x^2 / 2, to (x^2 / 2 + 8) u.
The smallest subnormal times what it is multiplied by is added for values that are subnormal."""
import math

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import assert_status_ok, require_gpu
from row_util import U, assert_within, gen

pytestmark = pytest.mark.gpu
A = fq.Activation
SMALL = 2.0 ** -148


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def reference(kind, x):
    """f, f' and their tolerances."""
    if kind == A.GELU:
        cdf = 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
        t = x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        f, df = x * cdf, cdf + t
        return f, df, 11 * U * f.abs(), 10 * U * cdf + (0.5 * x * x + 9) * U * t.abs()
    k = 2 * math.sqrt(2 / math.pi)
    z, dz, ez = (x, torch.ones_like(x), 0.0) if kind == A.SILU else (
        k * (x + 0.044715 * x ** 3), k * (1 + 3 * 0.044715 * x * x), 6.0)
    # exp(-|z|), not a difference from 1: accurate where it is small
    t = torch.exp(-z.abs())
    s, sc = torch.where(z >= 0, 1.0, t) / (1 + t), torch.where(z >= 0, t, 1.0) / (1 + t)
    moved = s * sc * ez * z.abs() * U
    f, df = x * s, s + x * s * sc * dz
    return f, df, 13 * U * f.abs() + x.abs() * moved, 12 * U * s + 36 * U * (x * s * sc * dz).abs() + moved * (1 + (x * dz).abs())


def arguments():
    g = gen(960)
    return torch.cat([torch.linspace(-15, 15, 60001, device="cuda"), torch.linspace(-110, 110, 22001, device="cuda"),
                      torch.randn(20000, generator=g, device="cuda"), torch.randn(2000, generator=g, device="cuda") * 1e-20])


@pytest.mark.parametrize("kind", list(A))
@pytest.mark.parametrize("cols", [104001, 4000])      # element by element, 16-byte accesses
def test_values_and_derivatives(kind, cols):
    x = arguments()[: 104001 if cols == 104001 else 104000].view(-1, cols)
    y = fq.gated_act(x, None, kind)[0]
    da = fq.gated_act_backward(torch.ones_like(x), kind, a=x)[0]
    b, dy = torch.full_like(x, 0.5), torch.full_like(x, 2.0)
    gated = fq.gated_act(x, b, kind)[0]
    dga, dgb = fq.gated_act_backward(dy, kind, a=x, b=b)
    assert_status_ok()
    xd = x.double()
    f, df, tf, td = reference(kind, xd)
    tf, td = tf + U * f.abs() + SMALL * (1 + xd.abs()), td + U * df.abs() + SMALL * (1 + xd.abs() ** 3)
    assert_within(y, f, tf, "f")
    assert_within(da, df, td, "f'")
    # powers of two change no digit
    assert_within(gated, 0.5 * f, 0.5 * tf + SMALL, "f b")
    assert_within(dga, df, td, "dy b f'")
    assert_within(dgb, 2.0 * f, 2.0 * tf, "dy f")


@pytest.mark.parametrize("kind", list(A))
def test_infinities_and_large_values(kind):
    x = torch.tensor([[float("inf"), 3e38, 1e20, 1e10, 200.0, -200.0, -1e10, -1e20, -3e38, 0.0, -0.0, float("nan")]], device="cuda")
    y, dx = fq.gated_act(x, None, kind)[0], fq.gated_act_backward(torch.ones_like(x), kind, a=x)[0]
    assert_status_ok()
    assert torch.equal(y[0, :5], x[0, :5]) and not bool(y[0, 5:11].any()) and bool(y[0, 11].isnan())
    assert bool((dx[0, 1:5] == 1).all()) and not bool(dx[0, 5:9].any()) and bool(dx[0, 11].isnan())
    assert bool((dx[0, 9:11] == 0.5).all())
