"""The binding's own checks, found on the host (no GPU needed)."""
import pytest
import torch

import fp4_precision_gemm_b200 as fq


@pytest.mark.parametrize("recipe", [fq.FP8Q_BLOCKWISE, fq.FP8Q_MXFP8, fq.FP8Q_PERTENSOR, fq.FP8Q_NVFP4])
def test_products_of_host_tensors_are_refused(recipe):
    """The kernels would be given addresses of the host."""
    a = torch.zeros((128, 256), dtype=torch.uint8)
    s, one = torch.ones((2, 128)), torch.ones(1)
    with pytest.raises(ValueError, match="CUDA device"):
        fq.gemm(a, a, recipe, a_scale=s, b_scale=s, a_global=one, b_global=one)
    with pytest.raises(ValueError, match="CUDA device"):
        fq.gemm(a, a, recipe, a_scale=s, b_scale=s, a_global=one, b_global=one, split_tail=False,
                out=torch.zeros((128, 128), dtype=torch.bfloat16))
