"""Matrices without elements are described whatever their strides: nothing else is wrong with these
tensors than that they are not on a GPU."""
import pytest
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from scaled_quantize_gemm_amax_gb300 import build as fqbuild


@pytest.mark.parametrize("shape", [(0, 64), (4, 0), (0, 0)])
def test_strides_of_empty_matrices(shape):
    fqbuild.build()
    x = torch.zeros(()).expand(shape)
    assert x.stride() == (0, 0)
    for call in (lambda: fq.layer_norm(x), lambda: fq.gated_act(x, x),
                 lambda: fq.layer_norm_backward(x, torch.zeros(shape[0]), x=x, mean=torch.zeros(shape[0])),
                 lambda: fq.fp8_layer_norm(x, None, None, 1e-5, x, None, None, fq.Format.E4M3, None, None, stream=0)):
        with pytest.raises(ValueError, match="a CUDA tensor is needed"):
            call()
