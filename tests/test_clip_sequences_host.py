"""What the gradients' norm and clipping take as a sequence, without a GPU: a tensor of the CPU is the last thing refused."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from scaled_quantize_gemm_amax_gb300 import build as fqbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    fqbuild.build()


def test_generators_are_taken():
    for call in (lambda g: fq.grad_norm(g), lambda g: fq.clip_grad_norm(g, 1.0), lambda g: fq.clip_grad_norm(g, 1.0, out=list(g))):
        with pytest.raises(ValueError, match="CUDA"):
            call([torch.ones(3), torch.ones(5)])
    for call in (lambda g: fq.grad_norm(g), lambda g: fq.clip_grad_norm(g, 1.0),
                 lambda g: fq.clip_grad_norm(g, 1.0, out=(torch.ones(3) for _ in range(2)))):
        with pytest.raises(ValueError, match="CUDA"):
            call(torch.ones(3) for _ in range(2))


def test_refusals_name_what_is_wrong():
    for grads, out in (([torch.ones(3)], []), ((torch.ones(3) for _ in range(2)), (torch.ones(3) for _ in range(1)))):
        with pytest.raises(ValueError, match="as many tensors"):
            fq.clip_grad_norm(grads, 1.0, out=out)
    for empty in ([], (), iter(())):
        with pytest.raises(ValueError, match="at least one"):
            fq.clip_grad_norm(empty, 1.0)
    with pytest.raises(TypeError, match="grads: a sequence"):
        fq.clip_grad_norm(3, 1.0)
    with pytest.raises(TypeError, match="out: a sequence"):
        fq.clip_grad_norm([torch.ones(3)], 1.0, out=3)


def test_a_limit_is_needed():
    """Without one nothing would be clipped, and nothing said."""
    for bad in (None, "1", [1.0]):
        with pytest.raises(TypeError):
            fq.clip_grad_norm([torch.ones(3)], bad)
