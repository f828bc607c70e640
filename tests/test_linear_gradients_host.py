"""The FP8 linear layer's gradients as autograd sees them, with plain products in the kernels' place."""
import pytest
import torch

from scaled_quantize_gemm_amax_gb300 import linear as L


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    def quantize(x, kind, fmt, delayed):
        return x.detach(), None, x.detach().t().contiguous(), None

    def gemm(a, fa, ra, sa, b, fb, rb, sb, c, out):
        c.copy_(a @ b.t())

    monkeypatch.setattr(L, "_quantize", quantize)
    monkeypatch.setattr(L, "fp8_scaled_gemm", gemm)


def test_a_second_derivative_is_refused():
    torch.manual_seed(2)
    x, w = torch.randn((4, 8), requires_grad=True), torch.randn((6, 8), requires_grad=True)
    y = L.fp8_linear(x, w)
    assert torch.allclose(y, x @ w.t())
    gx, gw = torch.autograd.grad(y.square().sum(), (x, w), create_graph=True)
    assert torch.allclose(gx, 2 * y @ w, atol=1e-5) and torch.allclose(gw, 2 * y.t() @ x, atol=1e-5)
    for g in (gx, gw):
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.square().sum().backward(retain_graph=True)
