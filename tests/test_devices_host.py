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
