"""Calls given a stream of their own: the memory of their results and workspaces, taken from torch's allocator,
is neither another stream's that still writes it when the call runs, nor another call's while the caller's stream
still reads it."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


def codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).mul_(60.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cuda()


def scales(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.exp2(torch.randn(shape, generator=g)).mul_(0.01).cuda()


def tensors(result):
    """The tensors of a call's result, without the columns that only pad a row of scales."""
    if isinstance(result, torch.Tensor):
        return [result]
    if isinstance(result, list):
        return [t for r in result for t in tensors(r)]
    return [t for t in result.values() if t is not None]


def grouped_calls(fq, seed):
    """name -> call(stream) of the calls around an expert layer, on tensors of this seed."""
    R, C = 600, 256                                            # multiples of 4: scales without padding
    a, b, sa, sb = codes((R, C), seed), codes((2, 256, C), seed + 1), scales((2, R), seed + 2), scales((2, 2, 2), seed + 3)
    x = workloads.normal_bf16((R, C), 1.0, seed + 4, device="cuda")
    w = torch.ones(C, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, 300, R], dtype=torch.int32, device="cuda")
    q = fq.quantize_1x128_grouped(x, offs)
    r = fq.norm_residual(x, x, w, w, w)
    y = torch.empty_like(x)
    return {
        "grouped rows": lambda s: fq.gemm(a, b, a_scale=sa, b_scale=sb, m_offsets=offs, stream=s),
        "grouped wgrad": lambda s: fq.gemm(q["q_col"], q["q_col"], layout=fq.FP8Q_WGRAD, a_scale=q["s_col"],
                                           b_scale=q["s_col"], m_offsets=offs, stream=s),
        "grouped quantizer": lambda s: fq.quantize_1x128_grouped(x, offs, rowwise=True, stream=s),
        "norm": lambda s: fq.norm_residual(x, x, w, w, w, quantize=True, stream=s),
        "norm backward": lambda s: fq.norm_residual_backward(x, x, x, r["h"], r["rstd_pre"], w, w, r["rstd_post"], w,
                                                             stream=s),
        "clip": lambda s: fq.clip_grad_norm([x], 1.0, out=[y], stream=s),
    }


GROUPED = ["grouped rows", "grouped wgrad", "grouped quantizer", "norm", "norm backward", "clip"]


def results_outlive_their_use(calls, others, name):
    side = torch.cuda.Stream()
    want = [t.clone() for t in tensors(calls[name](None))]
    torch.cuda.synchronize()
    got = tensors(calls[name](side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)                             # about a tenth of a second
    copies = [t.clone() for t in got]                          # the caller's stream reads them after that
    del got
    again = others[name](side)                                 # runs at once
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, copies))
    assert again is not None


@pytest.mark.parametrize("name", GROUPED)
def test_results_freed_while_the_callers_stream_reads_them(cuda_lib, name):
    results_outlive_their_use(grouped_calls(cuda_lib, 1), grouped_calls(cuda_lib, 11), name)
