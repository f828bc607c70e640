"""The package imports wherever torch does; what needs a GPU fails at the call."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_needs_no_cuda_names_of_torch():
    # a torch built without CUDA has none of its _C module's CUDA functions
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, n)\n"
            "import scaled_quantize_gemm_amax_gb300 as fq\n"
            "from scaled_quantize_gemm_amax_gb300 import blocks, linear\n"
            "assert fq.scale_shape(fq.Recipe.BLOCK_1x128, 4, 256) == ((4, 2), torch.float32)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
