"""The dispatch rule of the grouped products, without a GPU: what the GPU tests' cases take, and the argument checks."""
import ctypes

import pytest

import scaled_quantize_gemm_amax_gb300 as fq
from grouped_cases import DEPTH, MX, O, R, ROWS, SMS, T, segments, tiles
from scaled_quantize_gemm_amax_gb300 import build as fqbuild

INVALID, SHAPE, UNSUPPORTED = 1, 2, 4


@pytest.fixture(scope="module", autouse=True)
def lib():
    fqbuild.build()
    return fq.load_library()


def check(recipe, blocks, m, n, width, stages, third):
    capacity = 128 * sum(blocks)
    plan = fq.fp8_debug_grouped_plan(recipe, recipe, O.BF16, len(blocks), capacity, n, m, SMS)
    assert (plan["width"], plan["stages"]) == (width, stages), plan
    assert (tiles(blocks, m, n, width) > 2 * (SMS if width else SMS // 2)) == third
    # the output's type may cost the ring a stage, never the width
    assert fq.fp8_debug_grouped_plan(recipe, recipe, O.FP32, len(blocks), capacity, n, m, SMS)["width"] == width


@pytest.mark.parametrize("recipe,experts,blocks,n,k,width,stages,third", ROWS)
def test_rows(recipe, experts, blocks, n, k, width, stages, third):
    check(recipe, segments(experts, blocks), 0, n, width, stages, third)


@pytest.mark.parametrize("recipe,experts,blocks,m,n,width,stages,third", DEPTH)
def test_depth(recipe, experts, blocks, m, n, width, stages, third):
    check(recipe, segments(experts, blocks), m, n, width, stages, third)


def test_the_cases_leave_nothing_out():
    for cases in (ROWS, DEPTH):
        assert {c[-3] for c in cases if c[0] == T} == {0, 32, 64, 96, 128, 160, 192, 224, 256}
        assert {c[-3] for c in cases if c[0] == MX} == {0, 64, 128, 192, 256}
        assert {c[-2] for c in cases if c[0] == T and c[-3] == 0} == {5, 6}
        # narrower tiles are taken where no CTA has a second one
        assert {c[-3] for c in cases if c[0] == T and c[-1]} == {0, 128, 160, 192, 224, 256}
        assert {c[-3] for c in cases if c[0] == MX and c[-1]} == {0, 128, 192, 256}


def test_accumulators():
    for case, want in (((T, 5, 3, 4096), 2), ((MX, 5, 3, 4096), 1), ((MX, 40, 1, 1920), 2), ((MX, 500, 1, 256), 1), ((T, 3, 8, 3200), 2)):
        recipe, experts, blocks, n = case
        assert fq.fp8_debug_grouped_plan(recipe, recipe, O.BF16, experts, 128 * experts * blocks, n)["accumulators"] == want


def test_rejects(lib):
    plan = (ctypes.c_int64 * 3)()

    def f(ra=4, rb=4, out=0, experts=4, cap=256, m=0, n=128, sms=152, at=plan):
        return lib.fp8_debug_grouped_plan(ra, rb, out, experts, cap, m, n, sms, at)

    assert f() == 0 and f(ra=4, rb=6) == 0 and f(cap=0) == 0 and f(n=0) == 0
    for bad in (dict(at=None), dict(experts=0), dict(cap=-128), dict(m=-128), dict(n=-128), dict(sms=1), dict(out=2), dict(ra=7)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(ra=0), dict(ra=1, rb=2), dict(ra=int(R.MX_1x32), rb=int(R.MX_1x32))):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(cap=200), dict(m=64), dict(n=100), dict(experts=1025), dict(cap=2 ** 31)):
        assert f(**bad) == SHAPE, bad
