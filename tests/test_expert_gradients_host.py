"""Gradients of the differentiable RMS norm with a residual, without a GPU: none at all, and memory of their own."""
import itertools

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


# ways from leaves to an input of the norm
WAYS = {
    "leaf": lambda ts: ts[0],
    "product": lambda ts: ts[0] * 1.0,
    "sum": lambda ts: ts[0] + ts[1],
    "sum of a leaf": lambda ts: ts[0] + 0.0,
}


@pytest.mark.parametrize("used", ["y", "h", "both"])
@pytest.mark.parametrize("shape", [(6, 8), (2, 3, 8)])
@pytest.mark.parametrize("a,b", list(itertools.product(WAYS, WAYS)))
def test_gradients_do_not_share_memory(a, b, shape, used):
    """Both inputs have one gradient; every leaf behind them keeps it in memory of its own, so that one can be scaled or added to
    in place without another."""
    x0, x1, r0, r1 = ts = leaves(shape, shape, shape, shape)
    y, h = B.rms_norm(WAYS[a]((x0, x1)), None, WAYS[b]((r0, r1)))
    ry, rh = reference(WAYS[a]((x0, x1)), None, WAYS[b]((r0, r1)))
    dy, dh = torch.randn(shape, dtype=torch.float64), torch.randn(shape, dtype=torch.float64)
    pick = {"y": ((y, ry), (dy,)), "h": ((h, rh), (dh,)), "both": ((y, ry, h, rh), (dy, dh))}[used]
    outs, refs, grads = pick[0][::2], pick[0][1::2], pick[1]
    want = torch.autograd.grad(refs, ts, grads, allow_unused=True)
    torch.autograd.backward(outs, grads)
    have = [t for t in ts if t.grad is not None]
    for t, g in zip(ts, want):
        assert (t.grad is None) == (g is None)
        assert g is None or torch.allclose(t.grad, g)
    places = [t.grad.untyped_storage().data_ptr() for t in have] + [dy.untyped_storage().data_ptr(), dh.untyped_storage().data_ptr()]
    assert len(set(places)) == len(places)
    torch.autograd.backward(B.rms_norm(WAYS[a]((x0, x1)), None, WAYS[b]((r0, r1)))[:1], (dy,))   # added to what is there
    more = torch.autograd.grad(reference(WAYS[a]((x0, x1)), None, WAYS[b]((r0, r1)))[0], ts, dy, allow_unused=True)
    for t, g, m in zip(ts, want, more):
        assert g is None or torch.allclose(t.grad, g + m)


@pytest.mark.parametrize("shape", [(6, 8), (2, 3, 8)])
def test_outputs_can_be_changed_in_place(shape):
    """y is no part of what the backward pass needs."""
    x, res = leaves(shape, shape)
    y, h = B.rms_norm(x, None, res)
    y += 1
    y.sum().backward()
    ref = torch.autograd.grad(reference(x, None, res)[0].sum(), x)[0]
    assert torch.allclose(x.grad, ref) and torch.allclose(res.grad, ref)


@pytest.mark.parametrize("shape", [(6, 8), (2, 3, 8)])
def test_an_input_changed_before_the_backward_pass_is_noticed(shape):
    """Without a residual the backward pass needs x itself."""
    x, = leaves(shape)
    y = B.rms_norm(x)
    with torch.no_grad():
        x += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("used", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("way", ["leaf", "product", "sum of a leaf"])
@pytest.mark.parametrize("shape", [(6, 8), (2, 3, 8)])
def test_one_tensor_as_both_inputs(shape, way, used):
    x, = leaves(shape)
    grads = [g for g, u in zip((torch.randn(shape, dtype=torch.float64), torch.randn(shape, dtype=torch.float64)), used) if u]
    a = WAYS[way]((x,))
    torch.autograd.backward([t for t, u in zip(B.rms_norm(a, None, a), used) if u], grads)
    want, = torch.autograd.grad([t for t, u in zip(reference(x, None, x), used) if u], x, grads)
    assert torch.allclose(x.grad, want)


@pytest.mark.parametrize("residual", [False, True])
def test_inputs_that_are_copied_are_copied_once(residual, monkeypatch):
    """A transposed input is made contiguous for the forward pass; the backward pass takes that copy."""
    x, = leaves((8, 6))
    seen = []
    forward, backward = B._rms_norm, B._rms_norm_backward
    monkeypatch.setattr(B, "_rms_norm", lambda x, *a: seen.append(x.data_ptr()) or forward(x, *a))
    monkeypatch.setattr(B, "_rms_norm_backward", lambda dy, h, *a, **k: seen.append(h.data_ptr()) or backward(dy, h, *a, **k))
    res = torch.randn(6, 8, dtype=torch.float64) if residual else None
    y = B.rms_norm(x.t(), None, res)
    y = y[0] if residual else y
    dy = torch.randn(6, 8, dtype=torch.float64)
    got, = torch.autograd.grad(y, x, dy)
    want, = torch.autograd.grad(reference(x.t(), None, res)[0], x, dy)
    assert torch.allclose(got, want)
    assert seen[0] != x.data_ptr() and (residual or seen[1] == seen[0])
