"""Offsets that leave rows of A before the first expert or behind the last one: they break the rule (0 first, M
last), so the status word says so; the rows of no expert stay as they were and the others are computed."""
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


# in the kernel for few rows, and in the one for many
@pytest.mark.parametrize("M,offs", [(24, [0, 5, 5, 20]), (24, [3, 8, 8, 24]), (24, [2, 8, 9, 23]), (24, [0, 0, 0, 0]),
                                    (2000, [0, 700, 700, 1900]), (2000, [1, 700, 700, 2000]),
                                    (2000, [5, 700, 900, 1999]), (2000, [0, 0, 0, 0])], ids=str)
@pytest.mark.parametrize("layout", ["fprop", "dgrad"])
@pytest.mark.parametrize("acc", [False, True])
def test_rows_of_no_expert(cuda_lib, M, offs, layout, acc):
    fq = cuda_lib
    K, N, G = 256, 144, 3
    dgrad = layout == "dgrad"
    lay = fq.FP8Q_DGRAD if dgrad else fq.FP8Q_FPROP
    a, b, sa, sb = codes((M, K), 1), codes((G, N, K), 2), scales((2, M), 3), scales((G, 2, 2), 4)
    call = lambda o, out: fq.gemm(a, b, layout=lay, a_scale=sa, b_scale=sb, out=out, accumulate_fp32=acc,  # noqa: E731
                                  m_offsets=torch.tensor(o, dtype=torch.int32, device="cuda"))
    new = lambda: torch.full((M, N), 7.0, dtype=torch.float32 if acc else torch.bfloat16, device="cuda")  # noqa: E731
    assert fq.device_status() == fq.FP8Q_OK
    got = call(offs, new())
    assert fq.device_status() == fq.FP8Q_ERR_DEVICE_ARG
    assert fq.device_status() == fq.FP8Q_OK
    lo, hi = offs[0], offs[-1]
    assert bool((got[:lo] == 7.0).all()) and bool((got[hi:] == 7.0).all())
    # the same experts with the other rows given to the first and the last of them
    want = call([0] + offs[1:-1] + [M], new())
    assert fq.device_status() == fq.FP8Q_OK
    assert torch.equal(got[lo:hi], want[lo:hi])
