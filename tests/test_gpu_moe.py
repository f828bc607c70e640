"""Expert routing, dispatch and combine, against plain lists (whole numbers, exact) and 64-bit
sums.  Tolerances, u = 2^-24: a sum of k products (k + 1) u times the sum of their magnitudes, a
dot product of n terms (n + 2) u times it, for any order; one rounding to the output's type."""
import numpy as np
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import Guarded, assert_status_ok, host, require_gpu
from row_util import DTYPES, U, assert_within, gen, matrix, out_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def route_ref(ids, n_experts, align, capacity):
    lists = [[] for _ in range(n_experts)]
    flat = ids.reshape(-1).tolist()
    for i, e in enumerate(flat):
        if 0 <= e < n_experts:
            lists[e].append(i)
    offsets, pos, src = [0], [-1] * len(flat), [-1] * capacity
    for one in lists:
        for rank, i in enumerate(one):
            pos[i] = offsets[-1] + rank
            src[pos[i]] = i
        offsets.append(offsets[-1] + -(-len(one) // align) * align)
    return np.array(offsets, np.int32), np.array(pos, np.int32).reshape(ids.shape), np.array(src, np.int32)


def choices(tokens, k, n_experts, seed, drop=0.1, dtype=torch.int64):
    g = gen(seed)
    ids = torch.randint(0, n_experts, (tokens, k), generator=g, device="cuda")
    # a few experts get most of the choices, and some choices are dropped
    ids = torch.where(torch.rand((tokens, k), generator=g, device="cuda") < 0.4, ids // 3, ids)
    ids = torch.where(torch.rand((tokens, k), generator=g, device="cuda") < drop, -1, ids)
    return ids.to(dtype)


def check_route(ids, n_experts, align):
    r = fq.moe_route(ids, n_experts, align)
    assert_status_ok()
    offsets, pos, src = route_ref(host(ids), n_experts, align, r.src.numel())
    assert np.array_equal(host(r.offsets), offsets)
    assert np.array_equal(host(r.pos), pos)
    assert np.array_equal(host(r.src), src)
    return r


@pytest.mark.parametrize("tokens,k,n_experts", [(1, 1, 1), (1, 2, 8), (3, 8, 64), (31, 1, 5), (1000, 2, 8), (1024, 1, 3),
                                                (1025, 4, 1), (4097, 1, 256), (2047, 8, 64), (20000, 8, 128), (5000, 3, 1024),
                                                (70001, 2, 7)])
@pytest.mark.parametrize("align", [1, 128, 48])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_route(tokens, k, n_experts, align, dtype):
    check_route(choices(tokens, k, n_experts, tokens + k, dtype=dtype), n_experts, align)


def test_route_extremes():
    one = torch.zeros((5000, 2), dtype=torch.int32, device="cuda")
    check_route(one, 16, 128)                                    # every choice to one expert
    check_route(one + 15, 16, 128)                               # to the last
    check_route(one - 1, 16, 128)                                # every choice dropped: all segments empty
    far = torch.tensor([[2 ** 40, -2 ** 40, 1], [16, -1, 2 ** 32]], device="cuda")   # out of range in 64 bits, not wrapped
    check_route(far, 16, 1)
    r = check_route(torch.zeros((0, 2), dtype=torch.int64, device="cuda"), 4, 128)   # no tokens
    assert r.src.numel() == 0 and host(r.offsets).tolist() == [0] * 5
    # more room than needed: the rows past the last segment are marked as padding too
    ids = choices(700, 2, 8, 5)
    cap = fq.fp8_moe_capacity(700, 2, 8, 128) + 1000
    offsets, src = torch.empty(9, dtype=torch.int32, device="cuda"), torch.empty(cap, dtype=torch.int32, device="cuda")
    pos = torch.empty((700, 2), dtype=torch.int32, device="cuda")
    fq.fp8_moe_route(ids, 8, 128, offsets, pos, src)
    ref = route_ref(host(ids), 8, 128, cap)
    for a, b in zip((offsets, pos, src), ref):
        assert np.array_equal(host(a), b)


SHAPES = [(1, 2, 8, 4096, 1), (1, 1, 4, 7, 128), (37, 3, 5, 1000, 16), (129, 2, 8, 128, 128), (500, 8, 64, 256, 128),
          (64, 2, 8, 5003, 1), (300, 6, 16, 1024, 1), (40, 12, 40, 264, 8), (9, 2, 4, 20000, 1)]


def garbage_rows(r, ys):
    """NaN in the rows that no choice fills: nothing may read them."""
    ys = ys.clone()
    ys[r.src < 0] = float("nan")
    return ys


@pytest.mark.parametrize("tokens,k,n_experts,cols,align", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_dispatch_and_combine(tokens, k, n_experts, cols, align, dtype):
    dt = DTYPES[dtype]
    r = check_route(choices(tokens, k, n_experts, 700 + cols), n_experts, align)
    cap = r.src.numel()
    x = matrix(tokens, cols, dt, 701)
    xs = fq.moe_dispatch(x, r)
    src = r.src.long()
    ref = torch.where((src >= 0)[:, None], x[src.clamp(min=0) // k], torch.zeros((), dtype=dt, device="cuda"))
    assert torch.equal(xs, ref)

    ys = garbage_rows(r, matrix(cap, cols, dt, 702))
    w = torch.rand((tokens, k), generator=gen(703), device="cuda")
    w = torch.where(r.pos < 0, float("nan"), w)                  # a dropped choice's weight is not read
    kept = (r.pos >= 0)[..., None]
    rows = torch.where(kept, ys[r.pos.clamp(min=0).long()].double(), 0.0)
    for weights in (w, None):
        y = fq.moe_combine(ys, r, weights)
        terms = rows if weights is None else torch.where(kept, rows * w[..., None].double(), 0.0)
        y_ref = terms.sum(1)
        assert_within(y, y_ref, out_tol(y_ref, (k + 1) * U * terms.abs().sum(1), dt), "y")
    assert torch.equal(fq.moe_dispatch_backward(ys, r), y)
    assert_status_ok()


@pytest.mark.parametrize("tokens,k,n_experts,cols,align", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_backward(tokens, k, n_experts, cols, align, dtype):
    dt = DTYPES[dtype]
    r = check_route(choices(tokens, k, n_experts, 710 + cols), n_experts, align)
    dy, ys = matrix(tokens, cols, dt, 711), garbage_rows(r, matrix(r.src.numel(), cols, dt, 712))
    w = torch.rand((tokens, k), generator=gen(713), device="cuda")
    w = torch.where(r.pos < 0, float("nan"), w)
    dys, dw = fq.moe_combine_backward(dy, ys, r, w)
    assert_status_ok()
    src = r.src.long()
    at = src.clamp(min=0)
    ref = torch.where((src >= 0)[:, None], dy.double()[at // k] * w.reshape(-1)[at].double()[:, None], 0.0)
    assert_within(dys, ref, out_tol(ref, torch.zeros_like(ref), dt), "dys")
    terms = torch.where((r.pos >= 0)[..., None], ys[r.pos.clamp(min=0).long()].double() * dy.double()[:, None], 0.0)
    dw_ref = terms.sum(2)
    assert_within(dw, dw_ref, out_tol(dw_ref, (cols + 2) * U * terms.abs().sum(2), torch.float32), "dweights")
    # without weights: the copies of the rows
    plain, none = fq.moe_combine_backward(dy, ys, r)
    assert none is None and torch.equal(plain, fq.moe_dispatch(dy, r))


def test_gradient_against_differences():
    # combine is linear in ys and in the weights: a difference of any width is exact up to rounding
    r = check_route(choices(50, 3, 6, 720), 6, 8)
    ys, v = matrix(r.src.numel(), 96, torch.float32, 721), matrix(r.src.numel(), 96, torch.float32, 722)
    dy, w = matrix(50, 96, torch.float32, 723), torch.rand((50, 3), generator=gen(724), device="cuda")
    vw = torch.randn((50, 3), generator=gen(725), device="cuda")
    dys, dw = fq.moe_combine_backward(dy, ys, r, w)

    def loss(ys, w):
        rows = torch.where((r.pos >= 0)[..., None], ys.double()[r.pos.clamp(min=0).long()] * w.double()[..., None], 0.0)
        return (dy.double() * rows.sum(1)).sum()

    for grad, way, diff in ((dys, v, loss(ys.double() + v, w) - loss(ys.double() - v, w)),
                            (dw, vw, loss(ys, w.double() + vw) - loss(ys, w.double() - vw))):
        size = (grad.double() * way.double()).abs().sum()
        assert abs((grad.double() * way.double()).sum() - diff / 2) <= 1e-5 * size


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (16, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_alignments(pad, offset, dtype):
    dt, tokens, k, cols = DTYPES[dtype], 40, 2, 512
    r = check_route(choices(tokens, k, 4, 730), 4, 8)
    cap = r.src.numel()
    x, xs = matrix(tokens, cols, dt, 731, pad, offset), matrix(cap, cols, dt, 732, pad, offset)
    y, dys = matrix(tokens, cols, dt, 733, pad, offset), matrix(cap, cols, dt, 734, pad, offset)
    w, dw = torch.rand((tokens, k), device="cuda"), torch.empty((tokens, k), device="cuda")
    fq.fp8_moe_dispatch(x, r.pos, r.src, xs)
    assert torch.equal(xs, fq.moe_dispatch(x.contiguous(), r))
    fq.fp8_moe_combine(xs, r.pos, w, y)
    assert torch.equal(y, fq.moe_combine(xs.contiguous(), r, w))
    fq.fp8_moe_combine_backward(x, r.pos, r.src, w, xs, dys, dw)
    dense = fq.moe_combine_backward(x.contiguous(), xs.contiguous(), r, w)
    assert torch.equal(dys, dense[0])
    # the dots' order of summation may differ between the two accesses
    size = torch.where(r.pos >= 0, (x.double()[:, None] * xs.double()[r.pos.clamp(min=0).long()]).abs().sum(2), 0.0)
    assert bool(((dw.double() - dense[1].double()).abs() <= 2 * (cols + 2) * U * size).all())
    assert_status_ok()


def test_rows_out_of_range_are_reported_not_used():
    r = fq.moe_route(choices(16, 2, 4, 740, drop=0.0), 4, 8)
    bad = r.pos.clone()
    bad[3, 1], bad[5, 0] = r.src.numel(), -7
    ys = matrix(r.src.numel(), 256, torch.float32, 741)
    w = torch.ones((16, 2), device="cuda")
    for call in (lambda p: fq.moe_combine(ys, p, w), lambda p: fq.moe_dispatch(ys[:16], p),
                 lambda p: fq.moe_combine_backward(ys[:16], ys, p, w)[1]):
        got = call(fq.MoeRoute(r.offsets, bad, r.src))
        assert fq.fp8_get_device_status() == fq.Status.ERR_DEVICE_STATE
        assert fq.fp8_get_device_status() == fq.Status.OK
        good = call(r)
        assert_status_ok()
        if got.shape[0] == 16:      # the other tokens are as they were
            others = [t for t in range(16) if t not in (3, 5)]
            assert torch.equal(got[others], good[others])


def test_writes_stay_inside():
    tokens, k, n, cols = 77, 3, 6, 1001
    ids = choices(tokens, k, n, 750)
    cap = fq.fp8_moe_capacity(tokens, k, n, 16)
    g = {name: Guarded(shape, dt) for name, shape, dt in (
        ("offsets", (n + 1,), torch.int32), ("pos", (tokens, k), torch.int32), ("src", (cap,), torch.int32),
        ("xs", (cap, cols), torch.bfloat16), ("y", (tokens, cols), torch.bfloat16), ("dys", (cap, cols), torch.bfloat16),
        ("dw", (tokens, k), torch.float32))}
    t = {name: v.t for name, v in g.items()}
    x, w = matrix(tokens, cols, torch.bfloat16, 751), torch.rand((tokens, k), device="cuda")
    fq.fp8_moe_route(ids, n, 16, t["offsets"], t["pos"], t["src"])
    fq.fp8_moe_dispatch(x, t["pos"], t["src"], t["xs"])
    fq.fp8_moe_combine(t["xs"], t["pos"], w, t["y"])
    fq.fp8_moe_combine_backward(x, t["pos"], t["src"], w, t["xs"], t["dys"], t["dw"])
    assert_status_ok()
    for name, v in g.items():
        v.check(name)


def test_a_graph_on_another_stream():
    ids, x = choices(6000, 2, 8, 760), matrix(6000, 256, torch.bfloat16, 761)
    ref = fq.moe_route(ids, 8, 128)
    xs_ref = fq.moe_dispatch(x, ref)
    outs = [torch.empty_like(t) for t in (*ref, xs_ref)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):          # captures on a stream of its own
        fq.fp8_moe_route(ids, 8, 128, *outs[:3])
        fq.fp8_moe_dispatch(x, outs[1], outs[2], outs[3])
    for _ in range(2):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*ref, xs_ref), outs):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    r = check_route(torch.tensor([[0, 1, 2]], device="cuda"), 3, 1)
    ld = 1_200_000_000
    buf = torch.empty(2 * ld + 512, dtype=torch.bfloat16, device="cuda")
    xs = buf.as_strided((3, 512), (ld, 1))
    x = matrix(1, 512, torch.bfloat16, 770)
    fq.fp8_moe_dispatch(x, r.pos, r.src, xs)
    assert torch.equal(xs.contiguous(), x.expand(3, 512))
    assert torch.equal(fq.moe_combine(xs, r), fq.moe_combine(xs.contiguous(), r))
    assert_status_ok()
