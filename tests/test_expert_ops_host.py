"""Host-only checks of RMS norm, the grouped products and the gradients' norm: every refusal happens before any CUDA call."""
import ctypes

import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from scaled_quantize_gemm_amax_gb300 import build as fqbuild

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 4
FAKE = 0x10000          # an aligned address; never dereferenced by rejected calls
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    fqbuild.build()
    return fq.load_library()


def test_rms_norm_rejects(lib):
    def f(x=FAKE, rows=128, cols=128, ldx=128, dt=0, res=FAKE, ldr=128, w=FAKE, wdt=1, eps=1e-5, h=FAKE, ldh=128, y=FAKE, ldy=128,
          rstd=FAKE, recipe=0, fmt=0, scale=FAKE, amax=None, q=FAKE, ldq=128, s=FAKE):
        return lib.fp8_rms_norm(x, rows, cols, ldx, dt, res, ldr, w, wdt, eps, h, ldh, y, ldy, rstd, recipe, fmt, scale, amax, q, ldq,
                                s, None)

    for bad in (dict(x=None), dict(y=None, q=None), dict(rows=-1), dict(cols=-1), dict(dt=2), dict(wdt=-1), dict(fmt=2),
                dict(recipe=7), dict(recipe=-1), dict(eps=-1.0), dict(eps=NAN), dict(res=None), dict(scale=None),
                dict(recipe=1, s=None), dict(recipe=3, s=None), dict(recipe=1, amax=FAKE), dict(q=None, amax=FAKE)):
        assert f(**bad) == INVALID, bad
    assert f(recipe=2) == UNSUPPORTED
    for bad in (dict(ldx=127), dict(ldr=127), dict(ldh=127), dict(ldy=127), dict(ldq=127), dict(rows=2 ** 31), dict(ldx=2 ** 31),
                dict(recipe=3, cols=120), dict(recipe=4, rows=127), dict(recipe=4, cols=96), dict(recipe=6, rows=64),
                dict(cols=2 ** 31, ldx=2 ** 31)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(x=FAKE + 1), dict(dt=1, y=FAKE + 2), dict(w=FAKE + 2), dict(rstd=FAKE + 1), dict(res=FAKE + 1), dict(h=FAKE + 1),
                dict(recipe=1, s=FAKE + 2), dict(recipe=4, s=FAKE + 8), dict(amax=FAKE + 2), dict(scale=FAKE + 1)):
        assert f(**bad) == ALIGN, bad
    assert f(rows=0, x=None, y=None, q=None) == OK and f(cols=0, x=None, y=None) == OK


def test_rms_norm_backward_rejects(lib):
    def f(dy=FAKE, rows=4, cols=64, lddy=64, dt=0, h=FAKE, ldh=64, rstd=FAKE, dh=FAKE, lddh=64, w=FAKE, wdt=1, dx=FAKE, lddx=64,
          dw=FAKE, ws=FAKE, nbytes=1 << 30):
        return lib.fp8_rms_norm_backward(dy, rows, cols, lddy, dt, h, ldh, rstd, dh, lddh, w, wdt, dx, lddx, dw, ws, nbytes, None)

    for bad in (dict(dy=None), dict(dx=None), dict(rstd=None), dict(h=None), dict(ws=None), dict(dt=3), dict(wdt=2), dict(rows=-1),
                dict(cols=-1)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(lddy=63), dict(lddx=1), dict(ldh=63), dict(lddh=63), dict(nbytes=8), dict(rows=2 ** 31)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(dy=FAKE + 1), dict(ws=FAKE + 8), dict(dw=FAKE + 2), dict(dh=FAKE + 1), dict(dt=1, h=FAKE + 2)):
        assert f(**bad) == ALIGN, bad
    assert f(cols=0, dy=None) == OK
    assert f(rows=0, dy=None, dx=None, rstd=None, h=None, dw=None, ws=None) == OK


def test_workspaces(lib):
    for rows, cols in ((0, 128), (1, 1), (33, 4096), (10 ** 6, 12288)):
        assert fq.fp8_rms_norm_workspace(rows, cols) == 4 * cols * min(max(rows, 1), 304)
    n = ctypes.c_int64()
    assert lib.fp8_rms_norm_workspace(-1, 4, ctypes.addressof(n)) == INVALID
    assert lib.fp8_rms_norm_workspace(4, 4, None) == INVALID
    assert lib.fp8_rms_norm_workspace(4, 2 ** 31, ctypes.addressof(n)) == SHAPE
    assert 0 < fq.fp8_grad_norm_workspace(0) <= fq.fp8_grad_norm_workspace(1) <= fq.fp8_grad_norm_workspace(5000)
    assert lib.fp8_grad_norm_workspace(-1, ctypes.addressof(n)) == INVALID and lib.fp8_grad_norm_workspace(1, None) == INVALID


def test_grouped_gemm_rejects(lib):
    def f(a=FAKE, fa=0, ra=4, sa=FAKE, b=FAKE, fb=0, rb=4, sb=FAKE, count=1, offsets=FAKE, experts=4, cap=256, n=128, k=128, stacked=0,
          c=FAKE, out=0, tail=1):
        return lib.fp8_grouped_gemm(a, fa, ra, sa, b, fb, rb, sb, count, offsets, experts, cap, n, k, stacked, c, out, tail, None)

    for bad in (dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(offsets=None), dict(c=None), dict(fa=2), dict(fb=-1),
                dict(ra=7), dict(experts=0), dict(cap=-128), dict(n=-128), dict(k=-128), dict(stacked=2), dict(out=2),
                dict(ra=0, rb=0, count=2), dict(ra=0, rb=0, count=0)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(ra=0), dict(ra=1, rb=2), dict(ra=1, rb=1), dict(ra=3, rb=3), dict(rb=0)):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(cap=200), dict(n=64), dict(k=96), dict(experts=1025), dict(cap=2 ** 31), dict(n=2 ** 30), dict(k=2 ** 30, stacked=1),
                dict(cap=2 ** 30, n=2 ** 20)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(a=FAKE + 8), dict(b=FAKE + 1), dict(sa=FAKE + 8), dict(sb=FAKE + 4), dict(ra=0, rb=0, sa=FAKE + 2),
                dict(offsets=FAKE + 2), dict(c=FAKE + 8)):
        assert f(**bad) == ALIGN, bad
    assert f(cap=0, a=None, c=None) == OK and f(n=0, b=None, c=None) == OK


def test_grouped_wgrad_rejects(lib):
    def f(a=FAKE, fa=0, ra=4, sa=FAKE, b=FAKE, fb=0, rb=6, sb=FAKE, offsets=FAKE, experts=4, cap=256, m=128, n=128, c=FAKE, out=1):
        return lib.fp8_grouped_wgrad(a, fa, ra, sa, b, fb, rb, sb, offsets, experts, cap, m, n, c, out, None)

    for bad in (dict(a=None), dict(b=None), dict(sa=None), dict(sb=None), dict(offsets=None), dict(c=None), dict(fa=2), dict(rb=9),
                dict(experts=0), dict(cap=-128), dict(m=-128), dict(out=-1)):
        assert f(**bad) == INVALID, bad
    assert f(ra=1, rb=1) == UNSUPPORTED and f(ra=0) == UNSUPPORTED
    for bad in (dict(cap=200), dict(m=64), dict(n=100), dict(experts=2000), dict(m=2 ** 30), dict(m=2 ** 28, n=2 ** 20)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(a=FAKE + 8), dict(sb=FAKE + 8), dict(offsets=FAKE + 1), dict(c=FAKE + 4)):
        assert f(**bad) == ALIGN, bad
    assert f(m=0, a=None, c=None) == OK and f(n=0, c=None) == OK


def test_grad_norm_rejects(lib):
    def f(entries, max_norm=1.0, ws=FAKE, nbytes=1 << 20, norm=FAKE, n=None, clip=True):
        t = (fq.Gradient * max(len(entries), 1))(*[fq.Gradient(*e) for e in entries])
        n = len(entries) if n is None else n
        if clip:
            return lib.fp8_clip_grad_norm(ctypes.addressof(t), n, max_norm, ws, nbytes, norm, None)
        return lib.fp8_grad_norm(ctypes.addressof(t), n, ws, nbytes, norm, None)

    good = (FAKE, FAKE, 10, 1)
    for args in (dict(max_norm=-1.0), dict(max_norm=NAN), dict(ws=None), dict(norm=None), dict(n=-1)):
        assert f([good], **args) == INVALID, args
    for e in ((None, FAKE, 10, 1), (FAKE, None, 10, 1), (FAKE, FAKE, -1, 1), (FAKE, FAKE, 10, 2)):
        assert f([good, e]) == INVALID, e
    assert f([(FAKE, FAKE, 2 ** 40, 0)]) == SHAPE and f([(FAKE, FAKE, 2 ** 39, 0)] * 2) == SHAPE and f([good], nbytes=8) == SHAPE
    for e in ((FAKE + 2, FAKE, 10, 1), (FAKE, FAKE + 1, 10, 0)):
        assert f([e]) == ALIGN, e
    assert f([good], ws=FAKE + 4) == ALIGN and f([good], norm=FAKE + 2) == ALIGN
    assert f([(FAKE + 1, None, 10, 0)], clip=False) == ALIGN and f([(None, None, 10, 0)], clip=False) == INVALID


def test_helpers_refuse(lib):
    x, b = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.uint8)
    one, off = torch.ones(1), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fq.rms_norm(x)
    with pytest.raises(TypeError):
        fq.rms_norm(x.half())
    with pytest.raises(ValueError, match="residual"):
        fq.rms_norm(x, residual=torch.zeros(4, 127))
    with pytest.raises(ValueError, match="weight"):
        fq.rms_norm(x, torch.zeros(127))
    with pytest.raises(TypeError, match="rstd"):
        fq.rms_norm_backward(x, x, None)
    with pytest.raises(ValueError, match="h"):
        fq.rms_norm_backward(x, x.bfloat16(), torch.zeros(4))
    R, F = fq.Recipe, fq.Format
    with pytest.raises(ValueError, match="CUDA"):
        fq.grouped_gemm(b, F.E4M3, R.TENSOR, one, torch.zeros(256, 128, dtype=torch.uint8), F.E4M3, R.TENSOR, one, off)
    for bad in (dict(b=torch.zeros(255, 128, dtype=torch.uint8)), dict(b=torch.zeros(256, 64, dtype=torch.uint8)),
                dict(off=off.long()), dict(off=off[:1]), dict(a=x), dict(sa=one.double()), dict(sb=torch.ones(3)),
                dict(ra=R.MX_1x32_TILED)):
        with pytest.raises(ValueError):
            fq.grouped_gemm(bad.get("a", b), F.E4M3, bad.get("ra", R.TENSOR), bad.get("sa", one),
                            bad.get("b", torch.zeros(256, 128, dtype=torch.uint8)), F.E4M3, R.TENSOR, bad.get("sb", one),
                            bad.get("off", off))
    with pytest.raises(ValueError, match="columns"):
        fq.grouped_wgrad(b, F.E4M3, R.TENSOR, one, b[:, :64].contiguous(), F.E4M3, R.TENSOR, one, off)
    with pytest.raises(ValueError, match="CUDA"):
        fq.clip_grad_norm([x], 1.0)
    for grads, out in (([], None), ([x], []), ([x[:, ::2]], None)):
        with pytest.raises(ValueError):
            fq.clip_grad_norm(grads, 1.0, out=out)
    for grads in (x[0, 0], [x.half()], [None], 3):
        with pytest.raises(TypeError):
            fq.grad_norm(grads)
    with pytest.raises(TypeError):
        fq.clip_grad_norm([x], "1")
