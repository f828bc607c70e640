"""Differentiable row operators and an FP8 expert MLP block over them.

What stands between the FP8 linear layers of a transformer block (guide, "code changes":
the layers around the three GEMMs stay in BF16 / FP32), each as an autograd function over
the C ABI:

  layer_norm(x, weight, bias)    fp8_layer_norm / fp8_layer_norm_backward
  rms_norm(x, weight, residual)  fp8_rms_norm / fp8_rms_norm_backward
  gated_act(h)                   fp8_gated_act / fp8_gated_act_backward; h's halves are a and b
  moe_dispatch(x, route)         fp8_moe_dispatch / fp8_moe_combine
  moe_combine(ys, route, w)      fp8_moe_combine / fp8_moe_combine_backward

``checkpoint=Format.E4M3`` keeps what the backward pass needs (layer norm: the normalised
rows; activation: its inputs) as 8-bit codes with one multiplier per 128 columns instead of
the BF16 tensors; the forward values do not change.  A second derivative is an error.

``FP8MoEBlock`` is the pre-norm expert MLP of a transformer: norm, router, dispatch, two
FP8 linear layers per expert with a gated activation between them, combine, residual; with
``grouped`` the experts' layers are grouped products and no step waits for the routing.
Every operator runs in the library's kernels; torch does the router's small product and
top-k.  Leading dimensions are flattened; a tensor whose last dimension is not contiguous
or whose rows overlap (an expanded one) is copied.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (Activation, Format, MoeRoute, fp8_gated_act_backward, moe_route)
from . import gated_act as _gated_act
from . import layer_norm as _layer_norm
from . import layer_norm_backward as _layer_norm_backward
from . import moe_combine as _moe_combine
from . import moe_combine_backward as _moe_combine_backward
from . import moe_dispatch as _moe_dispatch
from . import moe_dispatch_backward as _moe_dispatch_backward
from . import rms_norm as _rms_norm
from . import rms_norm_backward as _rms_norm_backward
from .linear import FP8GroupedLinear, FP8Linear

__all__ = ["layer_norm", "rms_norm", "gated_act", "moe_dispatch", "moe_combine", "LayerNorm", "RMSNorm", "FP8MoEBlock"]


def _flat(x):
    """x as a matrix of rows of their own with a contiguous last dimension (an expanded one's rows share their memory)."""
    x = x.reshape(x.shape[:-1].numel(), x.shape[-1])   # -1 is ambiguous for rows of no columns
    dense = (x.stride(1) == 1 or x.shape[1] <= 1) and (x.stride(0) >= x.shape[1] or x.shape[0] <= 1)
    return x if dense else x.contiguous()


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, checkpoint):
        w = weight.detach() if weight is not None else None
        b = bias.detach() if bias is not None else None
        y, mean, rstd, q, s = _layer_norm(x, w, b, eps, checkpoint)
        if checkpoint is None:
            ctx.save_for_backward(w, rstd, x, mean)
        else:
            ctx.save_for_backward(w, rstd, q, s)
        ctx.meta = (checkpoint, weight is not None, bias.dtype if bias is not None else None)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w, rstd, a, b = ctx.saved_tensors
        checkpoint, has_weight, bias_dtype = ctx.meta
        saved = dict(x=a, mean=b) if checkpoint is None else dict(q=a, s=b, fmt=checkpoint)
        need = has_weight and ctx.needs_input_grad[1] or bias_dtype is not None and ctx.needs_input_grad[2]
        dx, dw, db = _layer_norm_backward(_flat(dy), rstd, w, param_grads=need, param_dtype=bias_dtype, **saved)
        return dx, dw if has_weight else None, db if bias_dtype is not None else None, None, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, checkpoint: Format | None = None):
    """Layer norm over the last dimension of x (bf16 or float32); weight and bias of one type, bf16 or float32."""
    return _LayerNormFn.apply(_flat(x), weight, bias, eps, checkpoint).reshape(x.shape)


class _RMSNormFn(torch.autograd.Function):
    # The inputs are flattened in here and both get one tensor as their gradient, as of torch's own sum: whoever keeps it sees
    # that others hold it too.  Views of it, which flattening outside would make, hide that.
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        w = weight.detach() if weight is not None else None
        rows = _flat(x)
        y, h, rstd, _, _ = _rms_norm(rows, w, _flat(residual) if residual is not None else None, eps)
        if residual is None:   # x itself, whose changes autograd notices, or the copy that was made of it
            h = x if rows.data_ptr() == x.data_ptr() else rows
        ctx.save_for_backward(w, h, rstd)
        ctx.has_residual, ctx.shape = residual is not None, x.shape
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        if dy is None and dh is None:   # what used the outputs has no gradient for them
            return None, None, None, None
        w, h, rstd = ctx.saved_tensors
        dw = None
        if dy is None:   # only h was used; its gradient may be kept elsewhere
            dx = dh.clone(memory_format=torch.contiguous_format)
        else:
            need = w is not None and ctx.needs_input_grad[1]
            dx, dw = _rms_norm_backward(_flat(dy), _flat(h), rstd, w, dh=_flat(dh) if dh is not None else None, param_grads=need)
        dx = dx.view(ctx.shape)
        return dx, dw, dx if ctx.has_residual else None, None


def rms_norm(x, weight=None, residual=None, eps: float = 1e-5):
    """RMS norm over the last dimension of x (bf16 or float32); weight bf16 or float32.

    With residual (like x) the norm of their sum h, rounded to x's type; returns (y, h) then."""
    if residual is None:
        return _RMSNormFn.apply(x, weight, None, eps).reshape(x.shape)
    if residual.shape != x.shape:
        raise ValueError(f"rms_norm: a residual of x's shape {tuple(x.shape)} is needed, not {tuple(residual.shape)}")
    y, h = _RMSNormFn.apply(x, weight, residual, eps)
    return y.reshape(x.shape), h.reshape(x.shape)


class _GatedActFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, act, gated, checkpoint):
        cols = h.shape[1] // 2 if gated else h.shape[1]
        a, b = (h[:, :cols], h[:, cols:]) if gated else (h, None)
        y, *codes = _gated_act(a, b, act, checkpoint)
        if checkpoint is None:
            ctx.save_for_backward(h)
        else:
            ctx.save_for_backward(*codes)
        ctx.meta = (act, gated, checkpoint, cols)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        act, gated, checkpoint, cols = ctx.meta
        dy = _flat(dy)
        dh = torch.empty((dy.shape[0], 2 * cols if gated else cols), dtype=dy.dtype, device=dy.device)
        da, db = (dh[:, :cols], dh[:, cols:]) if gated else (dh, None)
        a = b = qa = sa = qb = sb = None
        if checkpoint is None:
            h, = ctx.saved_tensors
            a, b = (h[:, :cols], h[:, cols:]) if gated else (h, None)
        else:
            qa, sa, qb, sb = ctx.saved_tensors
        fp8_gated_act_backward(dy, act, a, b, checkpoint or Format.E4M3, qa, sa, qb, sb, da, db)
        return dh, None, None, None


def gated_act(h, act: Activation = Activation.SILU, gated: bool = True, checkpoint: Format | None = None):
    """f(a) * b of the halves a, b of h's last dimension (gated), or f(h)."""
    if gated and h.shape[-1] % 2:
        raise ValueError(f"gated_act: the last dimension is split in two, but is {h.shape[-1]}")
    y = _GatedActFn.apply(_flat(h), act, gated, checkpoint)
    return y.reshape(*h.shape[:-1], y.shape[-1])


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, pos, src):
        ctx.save_for_backward(offsets, pos, src)
        return _moe_dispatch(x, MoeRoute(offsets, pos, src))

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        return _moe_dispatch_backward(_flat(dxs), MoeRoute(*ctx.saved_tensors)), None, None, None


def moe_dispatch(x, route: MoeRoute):
    """Every token's row of x [tokens, cols] at its choices' rows (0 in the rows that pad), differentiable in x."""
    return _DispatchFn.apply(_flat(x), *route)


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, offsets, pos, src):
        w = weights.detach().contiguous() if weights is not None else None
        ctx.save_for_backward(w, ys if w is not None else None, offsets, pos, src)
        ctx.shape = weights.shape if weights is not None else None
        return _moe_combine(ys, MoeRoute(offsets, pos, src), w)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w, ys, *route = ctx.saved_tensors
        dys, dw = _moe_combine_backward(_flat(dy), ys, MoeRoute(*route), w)
        return dys, dw.view(ctx.shape) if dw is not None else None, None, None, None


def moe_combine(ys, route: MoeRoute, weights=None):
    """Every token's choices' rows of ys [capacity, cols], summed with weights [tokens, k] float32 (None: 1)."""
    return _CombineFn.apply(_flat(ys), weights, *route)


class LayerNorm(torch.nn.Module):
    """Layer norm with float32 weight and bias; checkpoint: keep its normalised rows in 8 bits."""

    def __init__(self, cols: int, eps: float = 1e-5, checkpoint: Format | None = None, device=None):
        super().__init__()
        self.eps, self.checkpoint = eps, checkpoint
        self.weight = torch.nn.Parameter(torch.ones(cols, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(cols, device=device))

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps, self.checkpoint)


class RMSNorm(torch.nn.Module):
    """RMS norm with a float32 weight; with a residual it returns (y, x + residual)."""

    def __init__(self, cols: int, eps: float = 1e-5, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(cols, device=device))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps)


class FP8MoEBlock(torch.nn.Module):
    """x + sum over a token's k experts of w_e down_e(act(up_e(norm(x)))), a gated MLP an expert.

    hidden and ffn are multiples of 128 (the FP8 GEMM's tile); every expert's tokens are
    padded to 128 rows.  The experts' linear layers follow the fp8_autocast scope's recipe.
    checkpoint keeps the norm's rows (of a layer norm) and the activations' inputs in 8 bits.
    norm: "layer" or "rms".  grouped=False: a pair of FP8Linear an expert, and one host read of
    the segment starts per pass, which are the GEMMs' row counts.  grouped=True: two
    FP8GroupedLinear (per-tensor or MXFP8 recipes), without a host read, so that a pass can be
    captured into a CUDA graph (as torch asks of any backward pass, after a few eager steps on another
    stream and while nothing keeps an eager graph of the same parameters alive: drop its outputs first)."""

    def __init__(self, hidden: int, ffn: int, n_experts: int, k: int, act: Activation = Activation.SILU,
                 checkpoint: Format | None = Format.E4M3, device=None, norm: str = "layer", grouped: bool = False):
        super().__init__()
        if norm not in ("layer", "rms"):
            raise ValueError(f'norm: "layer" or "rms" is needed, not {norm!r}')
        self.n_experts, self.k, self.act, self.checkpoint, self.grouped = n_experts, k, act, checkpoint, grouped
        self.norm = RMSNorm(hidden, device=device) if norm == "rms" else LayerNorm(hidden, checkpoint=checkpoint, device=device)
        self.router = torch.nn.Parameter(torch.empty((n_experts, hidden), device=device))
        torch.nn.init.normal_(self.router, std=0.02)
        if grouped:
            self.up = FP8GroupedLinear(n_experts, hidden, 2 * ffn, device=device)
            self.down = FP8GroupedLinear(n_experts, ffn, hidden, device=device)
            return
        self.up = torch.nn.ModuleList(FP8Linear(hidden, 2 * ffn, device=device) for _ in range(n_experts))
        self.down = torch.nn.ModuleList(FP8Linear(ffn, hidden, device=device) for _ in range(n_experts))

    def forward(self, x):
        tokens = x.reshape(-1, x.shape[-1])
        n = self.norm(tokens)
        top = (n.float() @ self.router.t()).topk(self.k, dim=1)
        weights = torch.softmax(top.values, dim=1)
        route = moe_route(top.indices, self.n_experts, align=128)
        xs = moe_dispatch(n, route)
        if self.grouped:
            h = gated_act(self.up(xs, route.offsets), self.act, checkpoint=self.checkpoint)
            y = moe_combine(self.down(h, route.offsets), route, weights)
            return x + y.reshape(x.shape)
        starts = route.offsets.tolist()
        parts = []
        for e in range(self.n_experts):
            if starts[e] < starts[e + 1]:
                h = self.up[e](xs[starts[e]:starts[e + 1]])
                parts.append(self.down[e](gated_act(h, self.act, checkpoint=self.checkpoint)))
        if starts[-1] < xs.shape[0]:   # rows past the last segment, which no choice reads
            parts.append(xs.new_zeros((xs.shape[0] - starts[-1], xs.shape[1])))
        y = moe_combine(torch.cat(parts) if parts else xs, route, weights)
        return x + y.reshape(x.shape)
