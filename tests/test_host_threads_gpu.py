"""Calls from two host threads at once, each with its own stream and tensors and with another width than the
other's: what one thread's call sets up for its launch may not be undone by the other's.  Results are compared to
the bit with the same calls made by one thread."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


def norm_inputs(R, C, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda shape, dt, s: (torch.randn(shape, generator=g, device="cuda") * s).to(dt)  # noqa: E731
    return dict(y=rnd((R, C), B, 0.7), h=rnd((R, C), F, 1.5), w_pre=rnd((C,), F, 1.0), w_post=rnd((C,), F, 1.0),
                gate=rnd((C,), F, 0.5), dn=rnd((R, C), B, 1e-2), dh=rnd((R, C), F, 1e-2))


def forward(fq, x):
    return fq.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], alpha=0.9)


def backward(fq, x, r):
    return fq.norm_residual_backward(x["dn"], x["dh"], x["y"], r["h"], r["rstd_pre"], x["w_pre"], x["w_post"],
                                     r["rstd_post"], x["gate"], alpha=0.9)


# pairs that share a kernel: every forward width does, a backward width with those of as many columns per thread
PAIRS = [("forward", (256, 16384)), ("backward", (256, 4096)), ("backward", (8200, 16384))]


def both(work):
    """work(0) and work(1) in two threads that start together; their errors."""
    errors, start = [], threading.Barrier(2)

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                work(k)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


@pytest.mark.parametrize("what,widths", PAIRS)
def test_norms_of_two_widths(cuda_lib, what, widths):
    fq = cuda_lib
    jobs = [norm_inputs(3, C, 10 + C) for C in widths]
    saved = [forward(fq, x) for x in jobs]
    call = (lambda x, r: forward(fq, x)) if what == "forward" else (lambda x, r: backward(fq, x, r))
    alone = [call(x, r) for x, r in zip(jobs, saved)]
    torch.cuda.synchronize()
    got = [None, None]

    def work(k):
        for _ in range(300):
            got[k] = call(jobs[k], saved[k])

    assert not both(work)
    for a, g in zip(alone, got):
        assert a.keys() == g.keys()
        assert all(torch.equal(a[k], g[k]) for k in a)


@pytest.mark.parametrize("what,widths", PAIRS)
def test_c_calls_of_two_widths(cuda_lib, what, widths):
    """The C calls alone, which run beside one another outside Python's lock: every one of them is launched."""
    fq = cuda_lib
    L = fq.lib()
    jobs = [norm_inputs(1, C, 10 + C) for C in widths]
    saved = [forward(fq, x) for x in jobs]
    torch.cuda.synchronize()
    f32, bf16 = fq.FP8Q_FP32, fq.FP8Q_BF16
    p = lambda t: t.data_ptr()  # noqa: E731
    keep, args = [], []
    for C, x, r in zip(widths, jobs, saved):
        if what == "forward":
            o = [torch.empty_like(x["h"]), torch.empty_like(x["y"])]
            a = fq.NormArgs(1, C, f32, f32, 0.9, 1e-6, p(x["y"]), C, p(x["h"]), C, p(x["w_post"]), p(x["gate"]),
                            p(x["w_pre"]), p(o[0]), C, p(o[1]), C)
        else:
            n = fq.fp8q_norm_backward_workspace_bytes(1, C, f32)
            o = [torch.empty_like(x["dh"]), torch.empty_like(x["y"]), torch.empty((C,), device="cuda"),
                 torch.empty((n,), dtype=torch.uint8, device="cuda")]
            a = fq.NormBackwardArgs(1, C, f32, f32, 0.9, p(x["dn"]), C, p(x["dh"]), C, p(x["y"]), C, p(r["h"]), C,
                                    p(x["w_post"]), p(x["gate"]), p(x["w_pre"]), p(r["rstd_post"]), p(r["rstd_pre"]),
                                    p(o[0]), C, p(o[1]), C, None, None, p(o[2]), p(o[3]), n)
        keep.append(o)
        args.append(a)
    entry = L.fp8q_norm_residual if what == "forward" else L.fp8q_norm_residual_backward
    status = [set(), set()]

    def work(k):
        ref, stream = ctypes.byref(args[k]), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        for _ in range(40):
            for _ in range(500):
                status[k].add(entry(ref, stream))
            torch.cuda.current_stream().synchronize()

    assert not both(work)
    assert status == [{fq.FP8Q_OK}, {fq.FP8Q_OK}]
