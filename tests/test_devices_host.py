"""Which GPU a call runs on, checked without one: tensors that stand for memory of several GPUs
(no storage behind them) and a stand-in for the current device."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import scaled_quantize_gemm_amax_gb300 as fq
from scaled_quantize_gemm_amax_gb300 import build as fqbuild

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")


def on(gpu):
    """empty(*shape, dtype) of that GPU."""
    def empty(*shape, dtype=torch.float32):
        with FakeTensorMode():
            return torch.empty(shape, dtype=dtype, device=f"cuda:{gpu}")
    return empty


def test_helpers_refuse_tensors_of_two_gpus():
    fqbuild.build()
    a, b = on(0), on(1)
    i32 = torch.int32
    route = fq.MoeRoute(b(9, dtype=i32), b(4, 2, dtype=i32), b(8, dtype=i32))
    for call in (lambda: fq.layer_norm(a(4, 64), b(64)), lambda: fq.layer_norm(a(4, 64), a(64), b(64)),
                 lambda: fq.layer_norm_backward(a(4, 64), b(4), x=a(4, 64), mean=a(4)),
                 lambda: fq.layer_norm_backward(a(4, 64), a(4), a(64), q=a(4, 64, dtype=torch.uint8), s=b(4, 1)),
                 lambda: fq.gated_act(a(4, 64), b(4, 64)),
                 lambda: fq.gated_act_backward(a(4, 64), a=b(4, 64)),
                 lambda: fq.gated_act_backward(a(4, 64), qa=a(4, 64, dtype=torch.uint8), sa=b(4, 1)),
                 lambda: fq.moe_dispatch(a(4, 64), route), lambda: fq.moe_combine(a(8, 64), route),
                 lambda: fq.moe_combine(b(8, 64), route, a(4, 2)),
                 lambda: fq.moe_combine_backward(b(4, 64), a(8, 64), route, b(4, 2))):
        with pytest.raises(ValueError, match="of one device"):
            call()


def test_entry_points_refuse_tensors_of_another_gpu(monkeypatch):
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or 0

    monkeypatch.setattr(fq, "load_library", lambda path=None: Library())
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    fq._several_gpus.cache_clear()
    try:
        here, there = on(1), on(0)
        bf16, u8 = torch.bfloat16, torch.uint8

        def amax(at, to):
            fq.fp8_amax(at(4, 128, dtype=bf16), to(1), stream=0)

        def cast(at, to):
            fq.fp8_cast_transpose(at(128, 128, dtype=bf16), fq.Recipe.BLOCK_1x128, fq.Format.E4M3, None, None,
                                  to(128, 128, dtype=u8), to(128, 1), to(128, 128, dtype=u8), to(128, 1), stream=0)

        def norm(at, to):
            fq.fp8_layer_norm(at(4, 128), None, None, 1e-5, to(4, 128), None, None, fq.Format.E4M3, None, None, stream=0)

        for call in (amax, cast, norm):
            for at, to in ((there, there), (here, there), (there, here)):
                with pytest.raises(ValueError):
                    call(at, to)
            assert not calls
            call(here, here)
            assert len(calls) == 1
            calls.clear()
    finally:
        fq._several_gpus.cache_clear()
