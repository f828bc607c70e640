"""Host-only checks of the row operators: every refusal happens before any CUDA call, sizes are
host arithmetic, and the binding refuses tensors it cannot describe."""
import ctypes

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from scaled_quantize_gemm_amax_gb300 import build as fqbuild

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
FAKE = 0x10000          # an aligned address; never dereferenced by rejected calls
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    fqbuild.build()
    return fq.load_library()


def test_layer_norm_rejects(lib):
    def f(x=FAKE, rows=4, cols=64, ldx=64, dt=0, w=FAKE, b=FAKE, wdt=1, eps=1e-5, y=FAKE, ldy=64, mean=None, rstd=None, fmt=0,
          q=None, ldq=64, s=None):
        return lib.fp8_layer_norm(x, rows, cols, ldx, dt, w, b, wdt, eps, y, ldy, mean, rstd, fmt, q, ldq, s, None)

    for bad in (dict(x=None), dict(y=None), dict(rows=-1), dict(cols=-1), dict(dt=2), dict(wdt=-1), dict(fmt=2), dict(eps=-1.0),
                dict(eps=NAN), dict(q=FAKE), dict(s=FAKE)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(ldx=63), dict(ldy=63), dict(q=FAKE, s=FAKE, ldq=63), dict(cols=2 ** 31, ldx=2 ** 31, ldy=2 ** 31),
                dict(rows=2 ** 31), dict(ldx=2 ** 31)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(x=FAKE + 1), dict(dt=1, y=FAKE + 2), dict(w=FAKE + 2), dict(mean=FAKE + 1), dict(rstd=FAKE + 2),
                dict(q=FAKE, s=FAKE + 2)):
        assert f(**bad) == ALIGN, bad
    assert f(rows=0, x=None, y=None) == OK and f(cols=0, x=None, y=None) == OK


def test_layer_norm_backward_rejects(lib):
    def f(dy=FAKE, rows=4, cols=64, lddy=64, dt=0, x=FAKE, ldx=64, mean=FAKE, rstd=FAKE, fmt=0, q=None, ldq=64, s=None, w=FAKE,
          wdt=1, dx=FAKE, lddx=64, dw=FAKE, db=FAKE, ws=FAKE, nbytes=1 << 30):
        return lib.fp8_layer_norm_backward(dy, rows, cols, lddy, dt, x, ldx, mean, rstd, fmt, q, ldq, s, w, wdt, dx, lddx, dw, db,
                                           ws, nbytes, None)

    for bad in (dict(dy=None), dict(dx=None), dict(rstd=None), dict(x=None), dict(mean=None), dict(q=FAKE, s=FAKE),
                dict(x=None, mean=None, q=FAKE), dict(x=None, q=FAKE, s=FAKE), dict(ws=None), dict(dt=3), dict(fmt=5),
                dict(rows=-1)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(lddy=63), dict(lddx=1), dict(ldx=63), dict(x=None, mean=None, q=FAKE, s=FAKE, ldq=63), dict(nbytes=8)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(dy=FAKE + 1), dict(ws=FAKE + 8), dict(dw=FAKE + 2), dict(wdt=0, db=FAKE + 1)):
        assert f(**bad) == ALIGN, bad
    assert f(cols=0, dy=None) == OK
    assert f(rows=0, dy=None, dx=None, rstd=None, x=None, mean=None, dw=None, db=None, ws=None) == OK


def test_layer_norm_workspace(lib):
    assert fq.fp8_layer_norm_workspace(0, 128) >= 2 * 4 * 128        # no rows still sets the gradients
    for rows, cols in ((1, 1), (33, 4096), (10 ** 6, 12288)):
        assert fq.fp8_layer_norm_workspace(rows, cols) == 8 * cols * min(max(rows, 1), 304)
    n = ctypes.c_int64()
    assert lib.fp8_layer_norm_workspace(-1, 4, ctypes.addressof(n)) == INVALID
    assert lib.fp8_layer_norm_workspace(4, 4, None) == INVALID
    assert lib.fp8_layer_norm_workspace(4, 2 ** 31, ctypes.addressof(n)) == SHAPE


def test_gated_act_rejects(lib):
    def f(a=FAKE, rows=4, cols=64, lda=64, dt=0, act=0, b=FAKE, ldb=64, y=FAKE, ldy=64, fmt=0, qa=None, sa=None, qb=None, sb=None,
          ldq=64):
        return lib.fp8_gated_act(a, rows, cols, lda, dt, act, b, ldb, y, ldy, fmt, qa, sa, qb, sb, ldq, None)

    for bad in (dict(a=None), dict(y=None), dict(act=3), dict(act=-1), dict(dt=2), dict(fmt=2), dict(rows=-1), dict(qa=FAKE),
                dict(sb=FAKE), dict(b=None, qb=FAKE, sb=FAKE)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(lda=63), dict(ldb=63), dict(ldy=63), dict(qa=FAKE, sa=FAKE, ldq=63)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(a=FAKE + 1), dict(dt=1, b=FAKE + 2), dict(qa=FAKE, sa=FAKE + 1)):
        assert f(**bad) == ALIGN, bad
    assert f(rows=0, a=None, y=None) == OK


def test_gated_act_backward_rejects(lib):
    def f(dy=FAKE, rows=4, cols=64, lddy=64, dt=0, act=0, a=FAKE, lda=64, b=FAKE, ldb=64, fmt=0, qa=None, sa=None, qb=None,
          sb=None, ldq=64, da=FAKE, ldda=64, db=FAKE, lddb=64):
        return lib.fp8_gated_act_backward(dy, rows, cols, lddy, dt, act, a, lda, b, ldb, fmt, qa, sa, qb, sb, ldq, da, ldda, db,
                                          lddb, None)

    codes = dict(qa=FAKE, sa=FAKE, qb=FAKE, sb=FAKE)
    for bad in (dict(dy=None), dict(da=None), dict(db=None), dict(a=None), dict(b=None), codes, dict(codes, a=None),
                dict(codes, b=None), dict(codes, a=None, b=None, sa=None), dict(codes, a=None, b=None, db=None), dict(act=7)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(lddy=63), dict(lddb=63), dict(ldda=63), dict(codes, a=None, b=None, ldq=63)):
        assert f(**bad) == SHAPE, bad
    assert f(dy=FAKE + 1) == ALIGN
    assert f(cols=0, dy=None) == OK


def test_moe_route_rejects(lib):
    def f(ids=FAKE, size=4, tokens=16, k=2, n=8, align=1, offsets=FAKE, pos=FAKE, src=FAKE, cap=32):
        return lib.fp8_moe_route(ids, size, tokens, k, n, align, offsets, pos, src, cap, None)

    for bad in (dict(ids=None), dict(size=2), dict(tokens=-1), dict(k=0), dict(n=0), dict(align=0), dict(offsets=None),
                dict(pos=None), dict(src=None)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(cap=31), dict(n=1025), dict(align=128, cap=128), dict(tokens=2 ** 30), dict(cap=2 ** 31)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(ids=FAKE + 2), dict(size=8, ids=FAKE + 4), dict(pos=FAKE + 1)):
        assert f(**bad) == ALIGN, bad


def test_moe_capacity():
    assert fq.fp8_moe_capacity(8192, 2, 8, 128) == (16384 + 8 * 127) // 128 * 128
    assert fq.fp8_moe_capacity(1, 1, 64, 128) == 128                 # one choice: one segment
    assert fq.fp8_moe_capacity(0, 2, 8, 128) == 0
    assert fq.fp8_moe_capacity(3, 2, 8, 1) == 6
    assert fq.fp8_moe_capacity(100000, 8, 256, 128) % 128 == 0
    with pytest.raises(fq.FP8Error):
        fq.fp8_moe_capacity(2 ** 31, 1, 8, 1)
    with pytest.raises(fq.FP8Error):
        fq.fp8_moe_capacity(2 ** 29, 2, 8, 2 ** 30)


def test_moe_rows_reject(lib):
    def dispatch(x=FAKE, tokens=4, cols=64, ldx=64, dt=0, k=2, pos=FAKE, src=FAKE, cap=8, xs=FAKE, ldxs=64):
        return lib.fp8_moe_dispatch(x, tokens, cols, ldx, dt, k, pos, src, cap, xs, ldxs, None)

    def combine(ys=FAKE, cap=8, cols=64, ldys=64, dt=0, tokens=4, k=2, pos=FAKE, w=FAKE, y=FAKE, ldy=64):
        return lib.fp8_moe_combine(ys, cap, cols, ldys, dt, tokens, k, pos, w, y, ldy, None)

    def backward(dy=FAKE, tokens=4, cols=64, lddy=64, dt=0, k=2, pos=FAKE, src=FAKE, w=FAKE, ys=FAKE, ldys=64, cap=8, dys=FAKE,
                 lddys=64, dw=FAKE):
        return lib.fp8_moe_combine_backward(dy, tokens, cols, lddy, dt, k, pos, src, w, ys, ldys, cap, dys, lddys, dw, None)

    for bad in (dict(x=None), dict(pos=None), dict(src=None), dict(xs=None), dict(k=0), dict(dt=2), dict(tokens=-1), dict(cap=-1)):
        assert dispatch(**bad) == INVALID, bad
    assert dispatch(ldx=63) == dispatch(ldxs=63) == dispatch(tokens=2 ** 30, k=2) == SHAPE
    assert dispatch(x=FAKE + 1) == dispatch(src=FAKE + 2) == dispatch(dt=1, xs=FAKE + 2) == ALIGN
    assert dispatch(cols=0, x=None, xs=None) == dispatch(tokens=0, cap=0, x=None, pos=None, src=None, xs=None) == OK
    for bad in (dict(ys=None), dict(pos=None), dict(y=None), dict(k=0), dict(tokens=-1)):
        assert combine(**bad) == INVALID, bad
    assert combine(ldys=63) == combine(ldy=63) == SHAPE
    assert combine(w=FAKE + 2) == combine(ys=FAKE + 1) == ALIGN
    assert combine(tokens=0, ys=None, pos=None, y=None) == OK
    for bad in (dict(ys=None), dict(dy=None), dict(dys=None)):
        assert backward(**bad) == INVALID, bad
    assert backward(ldys=63) == backward(lddy=63) == backward(lddys=63) == SHAPE
    assert backward(dw=FAKE + 2) == ALIGN


def test_binding_refuses_what_it_cannot_describe():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    args = dict(y=torch.empty_like(x), mean=None, rstd=None, fmt=0, q=None, s=None, stream=0)

    def norm(x=x, weight=w, bias=None, **k):
        fq.fp8_layer_norm(x, weight, bias, 1e-5, **dict(args, **k))

    for bad in (dict(x=x.t()), dict(x=x[0]), dict(weight=w[:63]), dict(weight=w.to(torch.bfloat16), bias=w),
                dict(y=torch.empty((4, 63), dtype=torch.bfloat16)), dict(y=torch.empty((4, 64))), dict(mean=torch.empty(3)),
                dict(q=torch.empty((4, 64), dtype=torch.uint8)), dict(rstd=torch.empty(4, dtype=torch.float64))):
        with pytest.raises(ValueError, match="^(?!a CUDA)"):
            norm(**bad)
    with pytest.raises(TypeError):
        norm(x=x.half())
    with pytest.raises(ValueError, match="CUDA tensor"):   # nothing else is wrong with these
        norm()
    with pytest.raises(ValueError, match="^(?!a CUDA)"):
        fq.fp8_gated_act(x, x[:, :32], 0, torch.empty_like(x), 0, None, None, None, None, stream=0)
    with pytest.raises(ValueError, match="^(?!a CUDA)"):
        fq.fp8_moe_route(torch.zeros((4, 2)), 8, 1, *[torch.empty(n, dtype=torch.int32) for n in (9, 8, 8)], stream=0)
    pos, src = torch.zeros((4, 2), dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="^(?!a CUDA)"):
        fq.fp8_moe_dispatch(x, pos[:3], src, torch.empty((8, 64), dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError, match="^(?!a CUDA)"):
        fq.fp8_moe_dispatch(x, pos, src, torch.empty((7, 64), dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError, match="^(?!a CUDA)"):
        fq.fp8_moe_combine(x, pos, torch.ones((4, 2), dtype=torch.float64), x, stream=0)


def test_helpers_refuse_what_they_cannot_describe(lib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    route = fq.MoeRoute(*[torch.zeros(n, dtype=torch.int32) for n in (9, (4, 2), 8)])
    for call, what in ((lambda: fq.layer_norm(x.t()), "x"), (lambda: fq.layer_norm(x[0]), "x"), (lambda: fq.layer_norm(x, w[:63]), "weight"),
                       (lambda: fq.layer_norm(x, w.bfloat16(), w), "bias"),
                       (lambda: fq.layer_norm_backward(x, w), "rstd"),
                       (lambda: fq.layer_norm_backward(x, w[:4], x=x.float(), mean=w[:4]), "x"),
                       (lambda: fq.layer_norm_backward(x, w[:4], q=x, s=w[:4]), "q"),
                       (lambda: fq.layer_norm_backward(x, w[:4], q=x.byte(), s=w[:3]), "q"),
                       (lambda: fq.gated_act(x, x[:, :32]), "b"), (lambda: fq.gated_act(x, x.float()), "b"),
                       (lambda: fq.gated_act_backward(x, qa=x.byte()), "qa"),
                       (lambda: fq.gated_act_backward(x, a=x[:2]), "a"),
                       (lambda: fq.moe_route(torch.zeros((4, 2)), 8), "experts"),
                       (lambda: fq.moe_route(torch.zeros(4, dtype=torch.int32), 8), "experts"),
                       (lambda: fq.moe_dispatch(x[:3], route), "pos"),
                       (lambda: fq.moe_combine_backward(x[:3], x, route), "pos")):
        with pytest.raises(ValueError, match=f"^{what}:"):
            call()
    for call in (lambda: fq.layer_norm(None), lambda: fq.layer_norm(3), lambda: fq.layer_norm(x.half()), lambda: fq.layer_norm(x, w.half()),
                 lambda: fq.layer_norm_backward(x, w[:4], param_dtype=torch.half),
                 lambda: fq.gated_act(x.double()), lambda: fq.moe_combine(x.int(), route)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: fq.layer_norm(x, w), lambda: fq.gated_act(x, x), lambda: fq.moe_route(torch.zeros((4, 2), dtype=torch.int64), 8),
                 lambda: fq.moe_dispatch(x, route), lambda: fq.moe_combine(x, route)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
