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


def test_current_stream_without_torchs_own_function(monkeypatch):
    """A torch that lacks the function that only gives the stream's handle still has its public form."""
    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        if hasattr(torch._C, name):
            monkeypatch.delattr(torch._C, name)
    assert fq._stream().value == 0x1234
    assert fq._stream(Stream()).value == 0x1234
    assert fq._on(torch.device("cuda", 0), None) is fq._HERE
