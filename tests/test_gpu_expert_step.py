"""RMS norm, the grouped products and the gradients' norm together, as a training step and a token's step use them."""
import math

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from expert_util import F, MX, O, R, product_tol, values
from gpu_util import assert_status_ok, require_gpu
from row_util import assert_within, gen, out_tol
from scaled_quantize_gemm_amax_gb300 import blocks as B
from scaled_quantize_gemm_amax_gb300 import linear as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def routed(tokens, k, experts, seed):
    logits = torch.randn((tokens, experts), generator=gen(seed), device="cuda")
    return fq.moe_route(logits.topk(k, 1).indices, experts, align=128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("recipe", [L.Float8CurrentScaling(), L.MXFP8BlockScaling(), L.Float8DelayedScaling()])
def test_grouped_linear(recipe, dtype):
    """The layer's three products against 64-bit products of the operands as the casts give them."""
    experts, k, n = 5, 256, 384
    route = routed(300, 2, experts, 1)
    starts = route.offsets.tolist()
    layer = L.FP8GroupedLinear(experts, k, n, device="cuda")
    xs = fq.moe_dispatch(normal(300, k, seed=2, dtype=dtype), route).requires_grad_(True)
    dy = normal(xs.shape[0], n, seed=3, dtype=dtype)
    dy[starts[-1]:] = 0
    states = {r: fq.DelayedScaling(16, f) for r, f in (("x", F.E4M3), ("w", F.E4M3), ("dy", F.E5M2))} \
        if isinstance(recipe, L.Float8DelayedScaling) else {}
    with L.fp8_autocast(fp8_recipe=recipe):
        y = layer(xs, route.offsets)
    y.backward(dy)
    assert_status_ok()
    kx, kw = L._kinds(recipe)
    fx, fdy = recipe.fwd_format, recipe.bwd_format
    qx, sx, qxt, sxt = L._quantize(xs.detach(), kx, fx, states.get("x"))
    qw, sw, qwt, swt = L._quantize(layer.weight.detach().view(experts * n, k), kw, fx, states.get("w"))
    qd, sd, qdt, sdt = L._quantize(dy, kx, fdy, states.get("dy"))
    a, w, d = values(qx, kx, fx, sx), values(qw, kw, fx, sw), values(qd, kx, fdy, sd)
    at, wt, dt = values(qxt, kx, fx, sxt), values(qwt, kw, fx, swt), values(qdt, kx, fdy, sdt)
    for e in range(experts):
        r = slice(starts[e], starts[e + 1])
        for got, p, q, depth, what in ((y[r], a[r], w[n * e:n * (e + 1)], k, "y"), (xs.grad[r], d[r], wt[:, n * e:n * (e + 1)], n, "dx"),
                                       (layer.weight.grad[e], dt[:, r], at[:, r], r.stop - r.start, "dw")):
            ref = p @ q.t()
            assert_within(got.detach(), ref, out_tol(ref, product_tol(p, q, depth, None), got.dtype), f"{what} {e}")
    assert bool((y[starts[-1]:] == 0).all()) and bool((xs.grad[starts[-1]:] == 0).all())


def chain(block, x, recipe):
    """The block's forward pass by the public calls, with what its backward pass takes."""
    kx, kw = L._kinds(recipe)
    f = recipe.fwd_format
    y, _, rstd, _, _ = fq.rms_norm(x, block.norm.weight.detach())
    top = (y.float() @ block.router.detach().t()).topk(block.k, 1)
    w = torch.softmax(top.values, 1)
    route = fq.moe_route(top.indices, block.n_experts, align=128)
    xs = fq.moe_dispatch(y, route)

    def product(rows, weight):
        q, s, _, _ = L._quantize(rows, kx, f, None)
        qw, sw, _, _ = L._quantize(weight.detach().reshape(-1, weight.shape[2]), kw, f, None)
        return fq.grouped_gemm(q, f, kx, s, qw, f, kw, sw, route.offsets)

    h = product(xs, block.up.weight)
    cols = h.shape[1] // 2
    a = fq.gated_act(h[:, :cols], h[:, cols:], block.act)[0]
    return x + fq.moe_combine(product(a, block.down.weight), route, w)


@pytest.mark.parametrize("recipe", [L.Float8CurrentScaling(), L.MXFP8BlockScaling()])
@pytest.mark.parametrize("tokens", [0, 1, 300])
def test_block_is_the_chain_of_its_operators(recipe, tokens):
    torch.manual_seed(5)
    block = B.FP8MoEBlock(256, 384, n_experts=6, k=2, checkpoint=None, device="cuda", norm="rms", grouped=True)
    x = normal(tokens, 256, seed=6)
    with L.fp8_autocast(fp8_recipe=recipe), torch.no_grad():
        got = block(x)
    assert torch.equal(got, chain(block, x, recipe))
    assert_status_ok()


@pytest.mark.parametrize("recipe", [L.Float8CurrentScaling(), L.MXFP8BlockScaling(), L.Float8DelayedScaling()])
@pytest.mark.parametrize("tokens", [0, 1])
def test_gradients_of_few_tokens(recipe, tokens):
    """No token gives no gradient, one token gradients of its two experts alone."""
    torch.manual_seed(8)
    block = B.FP8MoEBlock(256, 384, n_experts=6, k=2, device="cuda", norm="rms", grouped=True)
    x = normal(tokens, 256, seed=9).requires_grad_(True)
    with L.fp8_autocast(fp8_recipe=recipe):
        y = block(x)
    y.backward(normal(tokens, 256, seed=10))
    assert x.grad.shape == x.shape and bool(x.grad.isfinite().all())
    for w in (block.up.weight, block.down.weight):
        used = w.grad.abs().amax((1, 2)) > 0
        assert int(used.sum()) == 2 * tokens and bool(w.grad.isfinite().all())
    assert block.norm.weight.grad.shape == (256,) and bool((block.norm.weight.grad != 0).any()) == (tokens > 0)
    assert bool(block.router.grad.isfinite().all()) and bool((block.router.grad != 0).any()) == (tokens > 0)
    assert_status_ok()


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_block_against_an_expert_at_a_time(norm):
    """MXFP8 scales lie in the experts' own rows, so both forms of the block multiply the same codes."""
    torch.manual_seed(9)
    one = B.FP8MoEBlock(256, 256, n_experts=4, k=2, checkpoint=None, device="cuda", norm=norm)
    all_ = B.FP8MoEBlock(256, 256, n_experts=4, k=2, checkpoint=None, device="cuda", norm=norm, grouped=True)
    with torch.no_grad():
        all_.router.copy_(one.router)
        for e in range(4):
            all_.up.weight[e].copy_(one.up[e].weight)
            all_.down.weight[e].copy_(one.down[e].weight)
    x = normal(500, 256, seed=10)
    dy = normal(500, 256, seed=11)
    out = []
    for block in (one, all_):
        x.grad = None
        x.requires_grad_(True)
        with L.fp8_autocast(fp8_recipe=L.MXFP8BlockScaling()):
            y = block(x)
        y.backward(dy)
        ups = torch.stack([m.weight.grad for m in block.up]) if block is one else block.up.weight.grad
        downs = torch.stack([m.weight.grad for m in block.down]) if block is one else block.down.weight.grad
        out.append((y.detach(), x.grad.clone(), ups, downs, block.router.grad.clone(), block.norm.weight.grad.clone()))
        x.requires_grad_(False)
    assert_status_ok()
    # binary32 sums in another order may round to another bf16, and that to another 8-bit code: a code is off by up to
    # 2^-3 of its value, and one value in a hundred at most lies so near a border
    for a, b, what in zip(*out, ("y", "dx", "up", "down", "router", "norm")):
        off = float((a.double() - b.double()).norm() / a.double().norm())
        assert off <= 2.0 ** -3 * 0.1, f"{what}: {off}"


def test_a_training_step():
    """Forward, backward, clipping, in a captured graph: replayed on new data it gives what eager calls give."""
    torch.manual_seed(12)
    block = B.FP8MoEBlock(256, 384, n_experts=4, k=2, device="cuda", norm="rms", grouped=True)
    params = list(block.parameters())
    x, dy = normal(400, 256, seed=13), normal(400, 256, seed=14)

    def step():
        with L.fp8_autocast(fp8_recipe=L.MXFP8BlockScaling()):
            y = block(x)
        grads = torch.autograd.grad(y, params, dy)
        was = [g.clone() for g in grads]
        norm = fq.clip_grad_norm(grads, 0.5)
        return y.detach(), was, grads, norm

    y, was, grads, norm = step()
    ref = math.sqrt(math.fsum(float(g.double().square().sum()) for g in was))
    assert abs(float(norm) - ref) <= 37 * 2.0 ** -24 * ref
    assert ref > 0.5 and abs(math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads)) - 0.5) < 1e-5
    del y, was, grads
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    x.copy_(normal(400, 256, seed=15))
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (got[0], *got[2], got[3])]
    eager = step()
    for a, b in zip(got, (eager[0], *eager[2], eager[3])):
        assert torch.equal(a, b)
    assert_status_ok()


def test_a_token_in_eight_bits():
    """One token through norm and linear layer: the norm's 8-bit rows are the product's operand (padded to its 128 rows)."""
    cols, n = 512, 256
    x, res, w = normal(1, cols, seed=20), normal(1, cols, seed=21), normal(cols, seed=22, dtype=torch.float32)
    wt = normal(n, cols, seed=23)
    qw, sw, _, _ = fq.cast_transpose(wt, R.BLOCK_128x128, F.E4M3, col=False)
    _, h, _, q, s = fq.rms_norm(x, w, res, recipe=R.BLOCK_1x128, keep_y=False)
    rows = torch.zeros((128, cols), dtype=torch.uint8, device="cuda")
    mult = torch.ones((128, cols // 128), device="cuda")
    rows[0], mult[0] = q[0], s[0]
    y = fq.scaled_gemm(rows, F.E4M3, R.BLOCK_1x128, mult, qw, F.E4M3, R.BLOCK_128x128, sw, O.FP32)[:1]
    a = values(q, R.BLOCK_1x128, F.E4M3, s)
    b = qw.view(torch.float8_e4m3fn).double() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    assert_within(y, a @ b.t(), 2.0 ** -23 * (cols + 64) * (a.abs() @ b.abs().t()), "y")
    assert torch.equal(h, x + res)
    assert_status_ok()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rms_norm_function(dtype):
    x, res, w = (normal(3, 7, 264, seed=30, dtype=dtype).requires_grad_(True), normal(3, 7, 264, seed=31, dtype=dtype).requires_grad_(True),
                 normal(264, seed=32, dtype=torch.float32).requires_grad_(True))
    dy, dh = normal(3, 7, 264, seed=33, dtype=dtype), normal(3, 7, 264, seed=34, dtype=dtype)
    y, h = B.rms_norm(x, w, res)
    torch.autograd.backward((y, h), (dy, dh))
    xd, wd = (x + res).detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    r = 1 / (xd.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    torch.autograd.backward((xd * r * wd, xd), (dy.double(), dh.double()))
    near = 1e-5 if dtype == torch.float32 else 2.0 ** -8
    for got, ref, tol in ((y, xd * r * wd, near), (x.grad, xd.grad, near), (res.grad, xd.grad, near), (w.grad, wd.grad, 1e-5)):
        assert float((got.double() - ref).norm() / ref.norm()) <= tol
    assert x.grad.data_ptr() != res.grad.data_ptr()
