"""Calls given a stream of their own: the memory of their results and workspaces, taken from torch's allocator,
is neither another stream's that still writes it when the call runs, nor another call's while the caller's stream
still reads it."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

GEMM = (1536, 3328, 6144)      # 78 tiles of 256 x 256 on 74 pairs of SMs


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


def plain_calls(fq, seed):
    """The same of the calls that are not grouped."""
    R, C = 512, 1024
    x = workloads.normal_bf16((R, C), 1.0, seed, device="cuda")
    w = workloads.normal_bf16((2, 256, C), 0.02, seed + 1, device="cuda")
    hist = torch.full((16,), 50.0, device="cuda")              # the largest stays, so every call has one scale
    M, N, K = GEMM
    a, b, sa, sb = codes((M, K), seed + 2), codes((N, K), seed + 3), scales((K // 128, M), seed + 4), scales(
        (N // 128, K // 128), seed + 5)
    assert fq.gemm_workspace_bytes(M, N, K) > 0                # its last wave of tiles is split
    delayed = lambda s: fq.quantize_tensor_delayed(x, hist, 0, stream=s)  # noqa: E731
    return {
        "gemm": lambda s: fq.gemm(a, b, a_scale=sa, b_scale=sb, stream=s),
        "1x128": lambda s: fq.quantize_1x128(x, colwise=True, stream=s),
        "128x128": lambda s: fq.quantize_128x128(x, stream=s),
        "128x128 grouped": lambda s: fq.quantize_128x128_grouped(w, stream=s),
        "multi": lambda s: fq.quantize_multi([("1x128", x, True, True), ("128x128", x, True, True)], stream=s),
        "mx32": lambda s: fq.quantize_mx32(x, colwise=True, stream=s),
        "tensor": lambda s: fq.quantize_tensor(x, stream=s),
        "tensor delayed": delayed,
        "nvfp4": lambda s: fq.rht16_quantize_sr(x, colwise=True, stream=s),
        "nvfp4 weights": lambda s: fq.quantize_nvfp4_2d16(x, stream=s),
    }


PLAIN = ["gemm", "1x128", "128x128", "128x128 grouped", "multi", "mx32", "tensor", "tensor delayed", "nvfp4",
         "nvfp4 weights"]
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


@pytest.mark.parametrize("name", PLAIN)
def test_plain_results_freed_while_the_callers_stream_reads_them(cuda_lib, name):
    results_outlive_their_use(plain_calls(cuda_lib, 1), plain_calls(cuda_lib, 11), name)


@pytest.mark.parametrize("name", PLAIN)
def test_results_in_memory_that_the_callers_stream_still_writes(cuda_lib, name):
    """Memory freed on the caller's stream, whose last kernel there has not run yet, is not handed to a call on
    another stream: its late write would land in that call's result or workspace."""
    fq = cuda_lib
    call = plain_calls(fq, 1)[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    sizes = [t.untyped_storage().nbytes() for t in tensors(call(None))]
    if name == "gemm":
        sizes.append(fq.gemm_workspace_bytes(*GEMM))
    torch.cuda.synchronize()
    old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda._sleep(200_000_000)                             # about a tenth of a second
    for t in old:
        t.fill_(0x7F)
    del old, t
    got = tensors(call(torch.cuda.Stream()))
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))


def test_a_stream_given_inside_a_capture(cuda_lib):
    """A captured step whose calls run on a forked stream of their own, replayed on new values."""
    fq = cuda_lib
    x = workloads.normal_bf16((512, 1024), 1.0, 1, device="cuda")
    qw = fq.quantize_128x128(workloads.normal_bf16((1024, 256), 0.02, 2, device="cuda"))
    side = torch.cuda.Stream()

    def step(s):
        q = fq.quantize_1x128(x, stream=s)
        return fq.gemm(q["q_row"], qw["q_t"], a_scale=q["s_row"], b_scale=qw["s"], stream=s)

    step(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        c = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for seed in (5, 6):
        x.copy_(workloads.normal_bf16((512, 1024), 1.0, seed, device="cuda"))
        g.replay()
        assert torch.equal(c, step(None))
