"""The wiring of the differentiable operators, without a GPU: what reaches the kernels, with plain
torch forms in the kernels' place that take what the entry points take and refuse the rest."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from scaled_quantize_gemm_amax_gb300 import blocks as B


def rows(x):
    """A matrix argument of an entry point: contiguous rows, a row stride of at least their length."""
    fq._rows(x, "x")
    assert x.shape[0] <= 1 or x.stride(0) >= x.shape[1], (x.shape, x.stride())
    return x.detach()


def plain_norm(x, w, b, eps, checkpoint):
    x = rows(x)
    mean, rstd = x.mean(1), 1 / (x.var(1, unbiased=False) + eps).sqrt()
    y = (x - mean[:, None]) * rstd[:, None]
    y = y if w is None else y * w
    return y if b is None else y + b, mean, rstd, None, None


def plain_norm_backward(dy, rstd, w, x, mean, param_grads, param_dtype):
    dy, x, r = rows(dy), rows(x), rstd[:, None]
    xh = (x - mean[:, None]) * r
    g = dy if w is None else dy * w
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0) if param_grads else None, dy.sum(0) if param_grads else None


def plain_act(a, b, act, checkpoint):
    a = rows(a)
    f = a * torch.sigmoid(a)
    return (f if b is None else f * rows(b)), None, None, None, None


def plain_act_backward(dy, act, a, b, fmt, qa, sa, qb, sb, da, db):
    dy, a = rows(dy), rows(a)
    s = torch.sigmoid(a)
    df = s * (1 + a * (1 - s))
    da.copy_(dy * df if b is None else dy * rows(b) * df)
    if b is not None:
        db.copy_(dy * a * s)


def plain_dispatch(x, route):
    at = route.src.long()
    return torch.where(at[:, None] >= 0, rows(x)[at.clamp(min=0) // route.pos.shape[1]], 0.0)


def plain_combine(ys, route, w=None):
    terms = torch.where(route.pos[..., None] >= 0, rows(ys)[route.pos.clamp(min=0).long()], 0.0)
    return (terms if w is None else terms * w.view(route.pos.shape)[..., None]).sum(1)


def plain_combine_backward(dy, ys, route, w):
    at = route.src.long().clamp(min=0)
    scale = torch.ones(route.pos.numel()) if w is None else w.reshape(-1)
    dys = torch.where(route.src[:, None] >= 0, rows(dy)[at // route.pos.shape[1]] * scale[at][:, None], 0.0)
    if w is None:
        return dys, None
    return dys, (plain_rows(ys, route) * rows(dy)[:, None]).sum(2)


def plain_rows(ys, route):
    return torch.where(route.pos[..., None] >= 0, rows(ys)[route.pos.clamp(min=0).long()], 0.0)


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    for name, f in (("_layer_norm", plain_norm), ("_layer_norm_backward", plain_norm_backward), ("_gated_act", plain_act),
                    ("fp8_gated_act_backward", plain_act_backward), ("_moe_dispatch", plain_dispatch),
                    ("_moe_dispatch_backward", plain_combine), ("_moe_combine", plain_combine),
                    ("_moe_combine_backward", plain_combine_backward)):
        monkeypatch.setattr(B, name, f)


# 3 tokens, 2 choices; one choice dropped, one row of padding
ROUTE = fq.MoeRoute(torch.tensor([0, 3, 6], dtype=torch.int32),
                    torch.tensor([[0, 3], [1, -1], [4, 2]], dtype=torch.int32),
                    torch.tensor([0, 2, 5, 1, 4, -1], dtype=torch.int32))


def operators():
    """name -> (the operator on an input of [n, 8] or [n, 16], its input's shape)."""
    torch.manual_seed(1)
    w = torch.rand((3, 2))
    return {"layer_norm": (lambda x: B.layer_norm(x, torch.full((8,), 1.5), torch.full((8,), 0.5)), (3, 8)),
            "gated_act": (B.gated_act, (3, 16)), "act": (lambda x: B.gated_act(x, gated=False), (3, 8)),
            "dispatch": (lambda x: B.moe_dispatch(x, ROUTE), (3, 8)),
            "combine": (lambda x: B.moe_combine(x, ROUTE, w), (6, 8)),
            "combine, no weights": (lambda x: B.moe_combine(x, ROUTE), (6, 8))}


NAMES = list(operators())


@pytest.mark.parametrize("name", NAMES)
def test_gradients_of_sums_over_rows(name):
    # the gradient of y.sum(0) is one row, expanded: its rows share their memory
    f, shape = operators()[name]
    x = torch.randn(shape, requires_grad=True)
    y = f(x)
    v = torch.randn(y.shape[1])
    got, = torch.autograd.grad((y.sum(0) * v).sum(), x, retain_graph=True)
    ref, = torch.autograd.grad(y, x, v.expand(y.shape).contiguous())
    assert torch.equal(got, ref)


@pytest.mark.parametrize("name", NAMES)
def test_expanded_inputs(name):
    f, shape = operators()[name]
    x = torch.randn((1, shape[1]), requires_grad=True)
    y = f(x.expand(shape))
    dy = torch.randn(y.shape)
    got, = torch.autograd.grad(y, x, dy)
    full = x.detach().expand(shape).contiguous().requires_grad_(True)
    y_ref = f(full)
    ref, = torch.autograd.grad(y_ref, full, dy)
    assert torch.equal(y, y_ref)
    assert torch.allclose(got, ref.sum(0, keepdim=True), atol=1e-5)


@pytest.mark.parametrize("name", NAMES)
def test_a_second_derivative_is_refused(name):
    # the backward passes have no derivatives of their own: a gradient that should carry a graph must not pass for one
    # that does
    f, shape = operators()[name]
    x = torch.randn(shape, requires_grad=True)
    g, = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


@pytest.mark.parametrize("name", ["dispatch", "combine", "combine, no weights"])
@pytest.mark.parametrize("changed", ["pos", "src"])
def test_a_routing_changed_before_the_backward_pass_is_noticed(name, changed, monkeypatch):
    monkeypatch.setitem(globals(), "ROUTE", fq.MoeRoute(*(t.clone() for t in ROUTE)))
    f, shape = operators()[name]
    y = f(torch.randn(shape, requires_grad=True))
    getattr(ROUTE, changed).fill_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("name", ["dispatch", "combine", "combine, no weights"])
def test_saved_tensor_hooks_see_the_routing(name):
    f, shape = operators()[name]
    seen = []

    def pack(t):
        seen.append(t)
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        f(torch.randn(shape, requires_grad=True))
    for t in (ROUTE.pos, ROUTE.src):
        assert any(s.data_ptr() == t.data_ptr() for s in seen)


@pytest.mark.parametrize("shape", [(3, 2), (6,), (1, 3, 2)])
def test_combine_weights_of_any_shape_have_a_gradient(shape):
    ys = torch.randn((6, 8))
    w = torch.rand(6)
    ref = w.view(3, 2).clone().requires_grad_(True)
    terms = plain_rows(ys, ROUTE) * ref[..., None]
    dy = torch.randn((3, 8))
    terms.sum(1).backward(dy)
    got = w.view(shape).clone().requires_grad_(True)
    B.moe_combine(ys, ROUTE, got).backward(dy)
    assert got.grad.shape == shape and torch.allclose(got.grad.view(3, 2), ref.grad)



def test_a_gradient_without_rows_that_is_expanded():
    # the gradient of y.sum() where y has no rows: strides 0, and contiguous() leaves it so
    for f in (lambda x: B.layer_norm(x), lambda x: B.gated_act(x, gated=False), B.gated_act):
        x = torch.randn((0, 8), requires_grad=True)
        f(x).sum().backward()
        assert x.grad.shape == (0, 8)


@pytest.mark.parametrize("shape", [(0, 8), (2, 0, 8), (3, 0), (2, 3, 0), (0,), (8,)])
def test_tensors_without_elements_and_without_leading_dimensions(shape):
    for f in (lambda x: B.layer_norm(x), lambda x: B.gated_act(x, gated=False), B.gated_act):
        x = torch.randn(shape, requires_grad=True)
        y = f(x)
        assert y.shape[:-1] == x.shape[:-1]
        y.sum().backward()
        assert x.grad.shape == x.shape
