"""The wiring of the differentiable RMS norm and of the grouped linear layer, without a GPU: plain torch forms stand in the
kernels' place."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from scaled_quantize_gemm_amax_gb300 import blocks as B
from scaled_quantize_gemm_amax_gb300 import linear as L


def rows(x):
    """A matrix argument of an entry point: contiguous rows, a row stride of at least their length."""
    fq._rows(x, "x")
    assert x.shape[0] <= 1 or x.stride(0) >= x.shape[1], (x.shape, x.stride())
    return x.detach()


def plain_norm(x, w, res, eps):
    h = rows(x) if res is None else rows(x) + rows(res)
    rstd = 1 / (h.square().mean(1) + eps).sqrt()
    y = h * rstd[:, None]
    return y if w is None else y * w, None if res is None else h, rstd, None, None


def plain_norm_backward(dy, h, rstd, w, dh=None, param_grads=True):
    r = rstd[:, None]
    xh = rows(h) * r
    g = rows(dy) if w is None else rows(dy) * w
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    return dx if dh is None else dx + rows(dh), (rows(dy) * xh).sum(0) if param_grads else None


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    monkeypatch.setattr(B, "_rms_norm", plain_norm)
    monkeypatch.setattr(B, "_rms_norm_backward", plain_norm_backward)


def reference(x, w, res):
    h = x if res is None else x + res
    y = h / (h.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    return (y if w is None else y * w), h


def leaves(*shapes):
    torch.manual_seed(3)
    return [torch.randn(s, dtype=torch.float64, requires_grad=True) if s is not None else None for s in shapes]


@pytest.mark.parametrize("used", ["y", "h", "both"])
@pytest.mark.parametrize("weight", [True, False])
def test_gradients_with_a_residual(used, weight):
    x, res, w = leaves((2, 3, 8), (2, 3, 8), (8,) if weight else None)
    a, b = torch.randn(2, 3, 8), torch.randn(2, 3, 8)

    def total(y, h):
        return (y * a).sum() * (used != "h") + (h * b).sum() * (used != "y") if used == "both" else \
            (y * a).sum() if used == "y" else (h * b).sum()

    def grads(f):
        for t in (x, res, w):
            if t is not None:
                t.grad = None
        total(*f()).backward()
        return [t.grad for t in (x, res, w) if t is not None]

    got, ref = grads(lambda: B.rms_norm(x, w, res)), grads(lambda: reference(x, w, res))
    for g, r in zip(got, ref):
        assert (g is None) == (r is None) or bool((r == 0).all())
        if g is not None:
            assert torch.allclose(g, r)
    # x and the residual share a gradient, but not its memory: one may be scaled in place without the other
    if got[0] is not None:
        assert got[0].data_ptr() != got[1].data_ptr()


def test_gradients_without_a_residual():
    x, w = leaves((3, 8), (8,))
    dy = torch.randn(3, 8, dtype=torch.float64)
    y = B.rms_norm(x, w)
    got = torch.autograd.grad(y, (x, w), dy)
    ref = torch.autograd.grad(reference(x, w, None)[0], (x, w), dy)
    assert all(torch.allclose(a, b) for a, b in zip(got, ref))


def test_expanded_inputs_and_gradients():
    x, res = leaves((1, 8), (1, 8))
    y, h = B.rms_norm(x.expand(3, 8), None, res.expand(3, 8))
    ry, rh = reference(x.expand(3, 8), None, res.expand(3, 8))
    assert torch.allclose(y, ry) and torch.allclose(h, rh)
    v = torch.randn(8, dtype=torch.float64)
    got = torch.autograd.grad((y.sum(0) * v).sum() + h.sum(), (x, res))
    ref = torch.autograd.grad((ry.sum(0) * v).sum() + rh.sum(), (x, res))
    assert all(torch.allclose(a, b) for a, b in zip(got, ref))


def test_a_second_derivative_is_refused():
    x, w = leaves((3, 8), (8,))
    g, = torch.autograd.grad(B.rms_norm(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


def test_h_changed_before_the_backward_pass_is_noticed():
    x, res = leaves((3, 8), (3, 8))
    y, h = B.rms_norm(x, None, res)
    with torch.no_grad():
        h += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("shape", [(0, 8), (2, 0, 8), (3, 0), (0,), (8,)])
def test_tensors_without_elements_and_without_leading_dimensions(shape):
    x, res = leaves(shape, shape)
    y, h = B.rms_norm(x, None, res)
    assert y.shape == x.shape and h.shape == x.shape
    (y.sum() + h.sum()).backward()
    assert x.grad.shape == x.shape and res.grad.shape == x.shape


def test_refusals():
    x = torch.randn(3, 8)
    with pytest.raises(ValueError, match="residual"):
        B.rms_norm(x, None, torch.randn(1, 8))
    with pytest.raises(ValueError, match="norm"):
        B.FP8MoEBlock(128, 128, 2, 1, norm="none")
    layer = L.FP8GroupedLinear(2, 128, 256)
    assert layer.weight.shape == (2, 256, 128)
    offsets = torch.zeros(3, dtype=torch.int32)
    with L.fp8_autocast(fp8_recipe=L.Float8BlockScaling()), pytest.raises(TypeError, match="blockwise"):
        layer(torch.zeros(128, 128), offsets)
    with L.fp8_autocast(fp8_recipe=L.MXFP8BlockScaling()):
        for xs, off in ((torch.zeros(128, 64), offsets), (torch.zeros(2, 128, 128), offsets), (torch.zeros(128, 128), offsets[:2])):
            with pytest.raises(ValueError):
                layer(xs, off)
    block = B.FP8MoEBlock(128, 256, 4, 2, norm="rms", grouped=True)
    assert {n: tuple(p.shape) for n, p in block.named_parameters()} == {
        "norm.weight": (128,), "router": (4, 128), "up.weight": (4, 512, 128), "down.weight": (4, 128, 256)}
