"""The differentiable operators on tensors whose rows share their memory: gradients of sums over
rows and expanded inputs give, bit for bit, what dense tensors give."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from gpu_util import assert_status_ok, require_gpu
from row_util import DTYPES, gen
from scaled_quantize_gemm_amax_gb300 import blocks as B

pytestmark = pytest.mark.gpu
TOKENS, COLS = 65, 264


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(*shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def operator(name):
    """The operator and its input's rows and columns."""
    route = fq.moe_route(torch.randint(-1, 6, (TOKENS, 3), generator=gen(900), device="cuda"), 6, 16)
    w = torch.rand((TOKENS, 3), generator=gen(901), device="cuda")
    return {"layer_norm": (lambda x: B.layer_norm(x, w.reshape(-1)[:1].expand(COLS).contiguous()), TOKENS, COLS),
            "layer_norm, 8 bits": (lambda x: B.layer_norm(x, checkpoint=fq.Format.E4M3), TOKENS, COLS),
            "gated_act": (B.gated_act, TOKENS, 2 * COLS),
            "gated_act, 8 bits": (lambda x: B.gated_act(x, checkpoint=fq.Format.E4M3), TOKENS, 2 * COLS),
            "act": (lambda x: B.gated_act(x, gated=False), TOKENS, COLS),
            "dispatch": (lambda x: B.moe_dispatch(x, route), TOKENS, COLS),
            "combine": (lambda x: B.moe_combine(x, route, w), route.src.numel(), COLS),
            "combine, no weights": (lambda x: B.moe_combine(x, route), route.src.numel(), COLS)}[name]


NAMES = ["layer_norm", "layer_norm, 8 bits", "gated_act", "gated_act, 8 bits", "act", "dispatch", "combine",
         "combine, no weights"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_expanded_gradients_and_inputs(name, dtype):
    f, rows, cols = operator(name)
    x = normal(rows, cols, seed=902, dtype=DTYPES[dtype]).requires_grad_(True)
    y = f(x)
    v = normal(y.shape[1], seed=903, dtype=y.dtype)
    got, = torch.autograd.grad(y, x, v.expand(y.shape), retain_graph=True)
    ref, = torch.autograd.grad(y, x, v.expand(y.shape).contiguous())
    assert torch.equal(got, ref)
    one = normal(cols, seed=904, dtype=DTYPES[dtype])
    assert torch.equal(f(one.expand(rows, cols)), f(one.expand(rows, cols).contiguous()))
    assert_status_ok()
