"""Global gradient norm over many tensors and clipping, against the same in 64 bits.

Tolerances.  Norm: eight squares are added in FP32 (nine roundings of at most 2^-24 of their
sum, all terms positive), the rest in FP64, the root halves the relative error and the result is
rounded to FP32: 5 * 2^-24 relative is over 9/2 + 1/2 steps.  Clipped values: the factor is
rounded once, the product once, and the factor carries the norm's error: (5 + 1 + 1) 2^-24, and
for BF16 half a step more, 2^-8 of the value."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

NORM = 5 * 2.0 ** -24
VALUE = {torch.float32: 7 * 2.0 ** -24, torch.bfloat16: 7 * 2.0 ** -24 + 2.0 ** -8}


def make(sizes, sigma=1.0, seed=0):
    """One tensor per (numel, dtype, offset): pieces of a NaN buffer, `offset` elements past an aligned address."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for n, dt, off in sizes:
        buf = torch.full((n + off + 16,), float("nan"), dtype=dt, device="cuda")
        t = buf[off:off + n]
        t.copy_(torch.randn(n, generator=g, device="cuda") * sigma)
        out.append((buf, t))
    return out


def reference(ts, max_norm, eps=1e-6):
    norm = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))
    return norm, min(1.0, max_norm / (norm + eps))


def check(ts, before, outs, norm, max_norm):
    ref, coef = reference(before, max_norm)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(float(norm) - ref) <= NORM * ref
    for b, o in zip(before, outs):
        want = b.double() * coef
        tiny = torch.finfo(torch.float32).tiny if coef != 1.0 else 0.0      # products below the normal range
        assert bool(((o.double() - want).abs() <= VALUE[b.dtype] * want.abs() + tiny).all())


F, B = torch.float32, torch.bfloat16
SETS = {
    "one element": [(1, F, 0)],
    "one bf16 at an odd address": [(1, B, 1)],
    "odd sizes and addresses": [(1, F, 3), (7, B, 5), (4096, F, 1), (8193, B, 7), (33, F, 2), (16384, B, 3), (0, F, 0),
                                (5, B, 0)],
    "chunk borders": [(4096, F, 0), (4097, F, 0), (8192, B, 0), (8191, B, 0), (4095, F, 1), (12288, F, 0)],
    "64 tensors": [(100 + k, F if k % 2 else B, k % 8) for k in range(64)],
    "65 tensors": [(100 + k, F if k % 2 else B, k % 8) for k in range(65)],
    "2100 tensors, three launches": [(k % 37, F if k % 3 else B, k % 5) for k in range(2100)],
    "large": [(3_000_001, F, 1), (5_000_003, B, 3)],
}


@pytest.mark.parametrize("place", ["in place", "out", "out at other addresses"])
@pytest.mark.parametrize("max_norm", [0.01, 1e9])
@pytest.mark.parametrize("name", SETS)
def test_clip(cuda_lib, name, max_norm, place):
    pieces = make(SETS[name], seed=len(name))
    ts = [t for _, t in pieces]
    before = [t.clone() for t in ts]
    if place == "in place":
        norm = cuda_lib.clip_grad_norm(ts, max_norm)
        outs, bufs = ts, [(b, off, t.numel()) for (b, t), (_, _, off) in zip(pieces, SETS[name])]
    else:
        shift = 0 if place == "out" else 1
        holders = [torch.full((n + off + 17,), float("nan"), dtype=dt, device="cuda") for n, dt, off in SETS[name]]
        outs = [h[off + shift:off + shift + n] for h, (n, dt, off) in zip(holders, SETS[name])]
        norm = cuda_lib.clip_grad_norm(ts, max_norm, out=outs)
        assert all(torch.equal(a, b) for a, b in zip(ts, before))          # inputs as they were
        bufs = [(h, off + shift, n) for h, (n, _, off) in zip(holders, SETS[name])]
    check(ts, before, outs, norm, max_norm)
    for buf, off, n in bufs:                                               # nothing written around the tensors
        assert bool(buf[:off].isnan().all()) and bool(buf[off + n:].isnan().all())


@pytest.mark.parametrize("sigma", [1e-30, 1e-25, 1e25, 3e37])
def test_squares_outside_fp32(cuda_lib, sigma):
    """Squares that overflow or underflow FP32 still give the norm."""
    ts = [t for _, t in make([(5000, F, 0), (3000, B, 1)], sigma=sigma, seed=3)]
    before = [t.clone() for t in ts]
    norm = cuda_lib.clip_grad_norm(ts, float("inf"))
    ref, _ = reference(before, float("inf"))
    if ref > 3.5e38:        # 3e37 * sqrt(8000) = 2.7e39 is past FP32's largest 3.403e38: nothing nearer than infinity
        assert float(norm) == math.inf
    else:
        assert abs(float(norm) - ref) <= NORM * ref
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    outs = [torch.empty_like(t) for t in ts]
    cuda_lib.clip_grad_norm(ts, 0.25 * ref, eps=0.0, out=outs)          # the factor comes from the 64-bit norm
    for b, o in zip(before, outs):
        want = b.double() * 0.25
        assert bool(((o.double() - want).abs() <= VALUE[b.dtype] * want.abs() + 1.2e-38).all())


def test_mixed_magnitudes_in_one_group(cuda_lib):
    """Tiny values beside large ones, zeros, and subnormals."""
    t = torch.tensor([1e-40, 0.0, 3.0, 1e-30, -4.0, 0.0, 1e-20, 0.0] * 9, device="cuda")
    ref, _ = reference([t], 1.0)
    assert abs(float(cuda_lib.clip_grad_norm([t], 1e9)) - ref) <= NORM * ref
    z = torch.zeros(1000, device="cuda")
    assert float(cuda_lib.clip_grad_norm([z], 1.0)) == 0.0 and bool((z == 0).all())


def test_nan_and_infinity(cuda_lib):
    a = torch.ones(100, device="cuda")
    b = torch.ones(100, device="cuda")
    b[7] = float("nan")
    assert math.isnan(float(cuda_lib.clip_grad_norm([a, b], 1.0)))
    assert bool(a.isnan().all()) and bool(b.isnan().all())
    for bad in (float("nan"), float("inf")):                   # no limit: the norm only, whatever it is
        a = torch.ones(100, device="cuda")
        a[3] = bad
        before = a.clone()
        assert not math.isfinite(float(cuda_lib.clip_grad_norm([a], math.inf)))
        assert torch.equal(a.view(torch.int32), before.view(torch.int32))
    a = torch.ones(100, device="cuda")
    a[3] = float("inf")
    assert float(cuda_lib.clip_grad_norm([a], 1.0)) == math.inf
    assert bool((a[:3] == 0).all()) and bool(a[3].isnan()) and bool((a[4:] == 0).all())


def test_zero_max_norm_and_zero_eps(cuda_lib):
    a = torch.randn(1000, device="cuda")
    cuda_lib.clip_grad_norm([a], 0.0)
    assert bool((a == 0).all())
    b = torch.randn(1000, device="cuda")
    before = b.clone()
    check([b], [before], [b], cuda_lib.clip_grad_norm([b], 0.5, eps=0.0), 0.5)


def test_shared_gradient_counts_twice_and_repeats_exactly(cuda_lib):
    g = torch.randn(70001, device="cuda")
    o = [torch.empty_like(g), torch.empty_like(g)]
    n1 = cuda_lib.clip_grad_norm([g, g], 1.0, out=o)
    check([g, g], [g, g], o, n1, 1.0)
    p = [torch.empty_like(g), torch.empty_like(g)]
    n2 = cuda_lib.clip_grad_norm([g, g], 1.0, out=p)
    assert float(n1) == float(n2) and torch.equal(o[0], p[0])


def test_more_than_four_gigabytes(cuda_lib):
    """Chunks and offsets past 32 bits: one tensor of 1.2e9 values and a small one."""
    a = torch.full((1_200_000_003,), 2.0 ** -10, device="cuda")
    b = torch.ones(5, dtype=B, device="cuda")
    a[-1] = 3.0
    norm = cuda_lib.clip_grad_norm([a, b], 1.0)
    ref = math.sqrt(1_200_000_002 * 2.0 ** -20 + 9.0 + 5.0)
    coef = 1.0 / (ref + 1e-6)
    assert abs(float(norm) - ref) <= NORM * ref
    for got, want in ((a[0], 2.0 ** -10 * coef), (a[1 << 30], 2.0 ** -10 * coef), (a[-2], 2.0 ** -10 * coef), (a[-1], 3 * coef)):
        assert abs(float(got) - want) <= VALUE[F] * want
    assert bool((a[:-1] == a[0]).all())


def test_graph_and_stream(cuda_lib):
    """Captured with many tensors and replayed on new values, beside an eager call on another stream."""
    ts = [torch.empty(1000 + k, device="cuda") for k in range(100)]
    other = [torch.randn(200000, device="cuda")]
    outs = [torch.empty_like(t) for t in ts]
    s = torch.cuda.Stream()
    fill = lambda seed: [t.copy_(torch.randn(t.shape, generator=torch.Generator("cuda").manual_seed(seed + k),  # noqa: E731
                                             device="cuda")) for k, t in enumerate(ts)]
    fill(0)
    cuda_lib.clip_grad_norm(ts, 1.0, out=outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = cuda_lib.clip_grad_norm(ts, 1.0, out=outs)
    for seed in (1000, 2000):
        fill(seed)
        torch.cuda.synchronize()
        was = other[0].clone()
        torch.cuda.synchronize()
        g.replay()
        eager = cuda_lib.clip_grad_norm(other, 3.0, stream=s)
        torch.cuda.synchronize()
        check(ts, ts, outs, norm, 1.0)
        check(other, [was], other, eager, 3.0)
