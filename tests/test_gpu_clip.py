"""The gradients' norm and clipping on the GPU, against 64-bit sums."""
import math

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import Guarded, require_gpu
from row_util import BF16, U, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _norm(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


# squares: a thread's 64 in binary32 chains of at most 65 additions, 5 over the warp, binary64 beyond; its root halves that, and the
# result is rounded once
NORM_TOL = 37 * U


def _check(grads, norm, outs, max_norm, was=None):
    ref = _norm(was if was is not None else grads)
    assert abs(float(norm) - ref) <= NORM_TOL * ref
    if outs is None:
        return
    by = min(1.0, max_norm / (ref + 1e-6))
    for g, o in zip(was if was is not None else grads, outs):
        want = g.double() * by
        tol = (want.abs() * (NORM_TOL + 4 * U)) + (want.abs() * BF16 if g.dtype == torch.bfloat16 else want.abs() * U)
        assert bool(((o.double() - want).abs() <= tol + 2.0 ** -133).all())


def _grads(sizes, dtypes, seed, sigma=1e-2, gap=0):
    """Tensors as views into one buffer a type, `gap` elements apart."""
    out, bufs, at = [], {}, {}
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        if dt not in bufs:
            total = sum(m + gap for j, m in enumerate(sizes) if dtypes[j % len(dtypes)] == dt)
            bufs[dt] = (torch.randn(total + 8, generator=gen(seed + len(bufs)), device="cuda") * sigma).to(dt)
            at[dt] = 0
        out.append(bufs[dt][at[dt]:at[dt] + n])
        at[dt] += n + gap
    return out


BOTH = [torch.bfloat16, torch.float32]
SIZES = [[1], [7], [4096], [1 << 20], [16384, 16385, 16383], [0, 5, 0], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10], [100003, 1, 65536, 30011],
         [777] * 300, [5] * 2000, [3 << 20, 17]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("dtypes", [BOTH[:1], BOTH[1:], BOTH], ids=["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("gap", [0, 3])
def test_norm_and_clip(sizes, dtypes, gap):
    grads = _grads(sizes, dtypes, 1, gap=gap)
    ref = _norm(grads)
    _check(grads, fq.grad_norm(grads), None, None)
    was = [g.clone() for g in grads]
    for max_norm in (ref * 0.3, ref * 3 + 1, 0.0):
        outs = [torch.full_like(g, 9.0) for g in grads]   # at other alignments than the views
        norm = fq.clip_grad_norm(grads, max_norm, out=outs)
        _check(grads, norm, outs, max_norm)
        assert all(torch.equal(g, w) for g, w in zip(grads, was))
    norm = fq.clip_grad_norm(grads, ref * 0.3)
    _check(grads, norm, grads, ref * 0.3, was)
    again = [g.clone() for g in grads]
    fq.clip_grad_norm(grads, ref + 1)     # not clipped: bit for bit as they were
    assert all(torch.equal(g, a) for g, a in zip(grads, again))


def test_neighbours_stay():
    """What lies between the gradients and around the outputs is not touched."""
    grads = _grads([33, 1000, 5, 20000], BOTH, 3, gap=5)
    outs = [Guarded(g.shape, g.dtype) for g in grads]
    buf = grads[0]._base.clone(), grads[1]._base.clone()
    fq.clip_grad_norm(grads, 0.01, out=[o.t for o in outs])
    for o in outs:
        o.check("out")
    assert torch.equal(grads[0]._base, buf[0]) and torch.equal(grads[1]._base, buf[1])
    fq.clip_grad_norm(grads, 0.01)
    for i, g in enumerate(grads):
        assert torch.equal(g, outs[i].t)
    for i in (0, 1):
        now, old = grads[i]._base, buf[i]
        ends = grads[i].numel(), grads[i].numel() + 5
        assert torch.equal(now[ends[0]:ends[1]], old[ends[0]:ends[1]])


@pytest.mark.parametrize("value", [1e-30, 1e-41, 3e30, 1e38])
def test_range(value):
    """Squares outside binary32's range count."""
    g = torch.full((70000,), value, device="cuda")
    ref = math.sqrt(70000) * float(g[0].double())
    norm = fq.grad_norm([g, torch.zeros(100, device="cuda")])
    if ref > torch.finfo(torch.float32).max:
        assert float(norm) == math.inf
    else:
        # a subnormal result has an absolute error of half its last place
        assert abs(float(norm) - ref) <= NORM_TOL * ref + 2.0 ** -150
    h = torch.full((70000,), 1.0, dtype=torch.bfloat16, device="cuda")
    h[7] = 3e30
    assert abs(float(fq.grad_norm([h])) / float(h[7]) - 1) <= NORM_TOL


def test_not_finite():
    for bad, dt in ((math.inf, torch.float32), (math.nan, torch.float32), (math.inf, torch.bfloat16), (math.nan, torch.bfloat16)):
        g = [torch.ones(5000, dtype=dt, device="cuda"), torch.ones(33, dtype=dt, device="cuda")]
        g[0][4321] = bad
        norm = fq.clip_grad_norm(g, 1.0)
        if math.isnan(bad):
            assert float(norm) != float(norm) and g[0].isnan().all() and g[1].isnan().all()
        else:
            assert float(norm) == math.inf and g[0][4321].isnan() and float(g[0][:4321].abs().max()) == 0 and (g[1] == 0).all()


def test_zero_and_infinite_limit():
    g = [torch.zeros(1000, device="cuda"), torch.zeros(3, dtype=torch.bfloat16, device="cuda")]
    assert float(fq.clip_grad_norm(g, 1.0)) == 0 and all((x == 0).all() for x in g)
    h = _grads([999], BOTH[:1], 5)
    was = h[0].clone()
    fq.clip_grad_norm(h, math.inf)
    assert torch.equal(h[0], was)


def test_dense_in_another_order():
    """A transposed gradient is dense: its elements are what counts."""
    g = torch.randn((70, 90), generator=gen(6), device="cuda").t()
    was = g.clone()
    norm = fq.clip_grad_norm([g], 1.0)
    _check([g], norm, [g], 1.0, [was])


def test_same_bits_every_time_and_captured():
    grads = _grads([100003, 77, 65536], BOTH, 7)
    outs = [torch.empty_like(g) for g in grads]
    first = fq.clip_grad_norm(grads, 0.5, out=outs).clone(), [o.clone() for o in outs]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = fq.clip_grad_norm(grads, 0.5, out=outs)
    for o in outs:
        o.fill_(4)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, first[0]) and all(torch.equal(a, b) for a, b in zip(outs, first[1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = fq.clip_grad_norm(grads, 0.5, out=outs, stream=side)
    side.synchronize()
    assert torch.equal(norm, first[0])


def test_through_the_c_names():
    grads = _grads([4097, 12, 300], BOTH, 8)
    outs = [torch.empty_like(g) for g in grads]
    ws = Guarded((fq.fp8_grad_norm_workspace(3),), torch.uint8)
    norm = torch.empty(1, device="cuda")
    fq.fp8_clip_grad_norm(grads, outs, 0.1, ws.t, norm)
    ws.check("workspace")
    want = [torch.empty_like(g) for g in grads]
    assert torch.equal(fq.clip_grad_norm(grads, 0.1, out=want), norm) and all(torch.equal(a, b) for a, b in zip(outs, want))
    fq.fp8_grad_norm(grads, ws.t, norm)
    ws.check("workspace")
    assert torch.equal(fq.grad_norm(grads), norm)
    fq.fp8_grad_norm([], ws.t, norm)
    assert float(norm) == 0


def test_refuses_shared_memory():
    b = torch.randn(1000, device="cuda")
    for grads, out in (([b[:600], b[500:]], None), ([b, b], None), ([b[:500], b[500:]], [b[500:], b[:500]]),
                       ([b[100:200]], [b[150:250]]), ([b[:10], b[10:20]], [torch.empty(10, device="cuda")] * 2)):
        was = b.clone()
        with pytest.raises(ValueError, match="share memory"):
            fq.clip_grad_norm(grads, 0.1, out=out)
        assert torch.equal(b, was)
    fq.clip_grad_norm([b[500:], b[:500]], 0.1, out=[b[500:], b[:500]])   # in place, in another order
    assert abs(float(fq.grad_norm([b, b])) - math.sqrt(2) * float(b.double().norm())) < 1e-5   # reading twice is fine


def test_a_write_is_seen_by_autograd():
    """A tensor that a backward pass still needs and that was clipped meanwhile is an error there, not a wrong gradient."""
    for out in (False, True):
        w, g, o = torch.randn(50, device="cuda", requires_grad=True), torch.randn(50, device="cuda"), torch.randn(50, device="cuda")
        loss = (w * (o if out else g)).sum()
        fq.grad_norm([g])
        fq.clip_grad_norm([g], 0.1, out=[o] if out else None)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():
        g = torch.ones(50, device="cuda")
    assert abs(float(fq.clip_grad_norm([g], 1.0)) - math.sqrt(50)) < 1e-5 and float(g[0]) < 0.2


def test_none_and_empty():
    """No gradient, and only ones without elements, at both sizes of a launch's table."""
    norm = torch.ones(1, device="cuda")
    ws = torch.empty(fq.fp8_grad_norm_workspace(200), dtype=torch.uint8, device="cuda")
    for n in (0, 1, 64, 200):
        grads = [torch.empty(0, device="cuda") for _ in range(n)]
        for _ in range(3):
            norm.fill_(1.0)
            fq.fp8_clip_grad_norm(grads, grads, 0.1, ws, norm)
            assert float(norm) == 0
            norm.fill_(1.0)
            fq.fp8_grad_norm(grads, ws, norm)
            assert float(norm) == 0
