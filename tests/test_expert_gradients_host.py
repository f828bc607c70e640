"""Gradients of the differentiable RMS norm with a residual, without a GPU: where there is none at all."""

import pytest
import torch

from scaled_quantize_gemm_amax_gb300 import blocks as B
from test_expert_blocks_host import leaves, plain, reference  # noqa: F401  (plain is a fixture)


class Dropped(torch.autograd.Function):
    """Passes its input on and no gradient back."""

    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, g):
        return None


@pytest.mark.parametrize("through", [lambda t: t, lambda t: t * 1.0], ids=["leaves", "results"])
@pytest.mark.parametrize("used", ["y", "h", "both"])
def test_no_gradient_at_all(used, through):
    """Where nothing comes back no input has a gradient, as of torch's own sum."""
    x, res, w = leaves((2, 8), (2, 8), (8,))
    y, h = B.rms_norm(through(x), w, through(res))
    out = {"y": Dropped.apply(y), "h": Dropped.apply(h), "both": Dropped.apply(y) + Dropped.apply(h)}[used]
    out.sum().backward()
    for t in (x, res, w):
        assert t.grad is None or bool((t.grad == 0).all())
