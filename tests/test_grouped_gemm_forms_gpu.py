"""Grouped gemm(): the same operands in any form that holds what the kernels read give the same result, to the
bit, in the kernel for few rows and in the other."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).mul_(60.0).clamp_(-448, 448).to(E4M3).view(torch.uint8).cuda()


def scales(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.exp2(torch.randn(shape, generator=g)).mul_(0.01).cuda()


def padded(t, rows, cols):
    """t (R, C) at the start of a larger tensor of NaN."""
    out = torch.full((t.shape[0] + rows, t.shape[1] + cols), float("nan"), device="cuda")
    out[:t.shape[0], :t.shape[1]] = t
    return out


@pytest.mark.parametrize("counts", [[5, 0, 11], [700, 0, 900]], ids=["few", "many"])
@pytest.mark.parametrize("layout", ["fprop", "dgrad"])
def test_forms_of_the_operands(cuda_lib, layout, counts):
    fq = cuda_lib
    G, M, K, N = len(counts), sum(counts), 384, 256
    dgrad = layout == "dgrad"
    lay = fq.FP8Q_DGRAD if dgrad else fq.FP8Q_FPROP
    offs = torch.tensor([0, counts[0], counts[0], M], dtype=torch.int32, device="cuda")
    a, b, sa = codes((M, K), 1), codes((G, N, K), 2), scales((K // 128, M), 3)
    sb = scales((G, 3, 2) if dgrad else (G, 2, 3), 4)
    flat = sb.view(-1, sb.shape[-1])
    call = lambda **kw: fq.gemm(**{**dict(a=a, b=b, layout=lay, a_scale=sa, b_scale=sb, m_offsets=offs), **kw})  # noqa: E731
    want = call()
    same = lambda got: torch.equal(got.view(torch.int16), want.view(torch.int16))  # noqa: E731
    assert same(call(a=a.view(E4M3), b=b.view(E4M3)))
    assert same(call(a=a.view(torch.int8), b=b.view(torch.int8)))
    assert same(call(b_scale=flat)) and same(call(b_scale=flat[None]))
    wide = padded(flat, 1, 5)
    assert same(call(b_scale=wide))
    assert same(call(b_scale=wide[:-1].reshape(G, -1, wide.shape[1])))
    assert same(call(b_scale=wide[:-1, :-5], ld_sb=wide.shape[1]))
    assert same(call(a_scale=padded(sa, 1, 4)))
    assert same(call(a_scale=padded(sa, 1, 4)[:-1, :-4], ld_sa=M + 4))
    assert same(call(a=torch.cat((a, codes((M, 128), 5)), 1), b=torch.cat((b, codes((G, N, 128), 6)), 2), K=K))
    assert same(call(b=torch.cat((b, codes((1, N, K), 7))), b_scale=torch.cat((sb, sb[:1]))))
    big = torch.full((M + 9, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    assert call(out=big) is big
    assert same(big[:M, :N].contiguous()) and bool((big[M:] == 7.0).all()) and bool((big[:, N:] == 7.0).all())
    acc, more = torch.ones((M, N), device="cuda"), torch.ones((M + 9, N + 24), device="cuda")
    call(out=acc, accumulate_fp32=True)
    call(out=more, accumulate_fp32=True)
    assert torch.equal(more[:M, :N], acc) and bool((more[M:] == 1.0).all()) and bool((more[:, N:] == 1.0).all())
    assert fq.device_status() == fq.FP8Q_OK


def test_forms_of_one_expert(cuda_lib):
    """One expert: its matrix may come out of a stack with gaps, its scales as one matrix."""
    fq = cuda_lib
    a, b, sa, sb = codes((300, 256), 1), codes((3, 256, 256), 2), scales((2, 300), 3), scales((1, 2, 2), 4)
    offs = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    want = fq.gemm(a, b[:1], a_scale=sa, b_scale=sb, m_offsets=offs)
    assert torch.equal(fq.gemm(a, b[::2][:1], a_scale=sa, b_scale=sb[0], m_offsets=offs), want)


def test_forms_of_wgrad_operands(cuda_lib):
    fq = cuda_lib
    counts, M, N = [130, 0, 60], 64, 96
    P = fq.fp8q_grouped_capacity(sum(counts), 3)
    offs = torch.tensor([0, 130, 130, 190], dtype=torch.int32, device="cuda")
    x, y, sx, sy = codes((M, P), 1), codes((N, P), 2), scales((P // 128, M), 3), scales((P // 128, N), 4)
    call = lambda **kw: fq.gemm(**{**dict(a=x, b=y, layout=fq.FP8Q_WGRAD, a_scale=sx, b_scale=sy, m_offsets=offs), **kw})  # noqa: E731
    want = call()
    assert torch.equal(call(a=x.view(E4M3), b=y.view(E4M3)), want)
    assert torch.equal(call(a_scale=padded(sx, 1, 4), b_scale=padded(sy, 1, 4)), want)
    assert torch.equal(call(a_scale=padded(sx, 0, 4)[:, :M], b_scale=padded(sy, 0, 4)[:, :N], ld_sa=M + 4, ld_sb=N + 4), want)
    assert fq.device_status() == fq.FP8Q_OK
