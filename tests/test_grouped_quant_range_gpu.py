"""The grouped 1x128 quantizer near the largest number of rows that 32-bit offsets can name."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


def test_one_expert_of_nearly_2_31_rows(cuda_lib):
    """2^31 - 64 rows of one expert, 16 columns: bands at the start, past 2^30 rows and at the ragged end against
    calls on those rows alone."""
    fq = cuda_lib
    torch.cuda.empty_cache()
    R, C = 2 ** 31 - 64, 16
    need = R * C * 2 + R * C + (8 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs 111 GB of device memory")
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    spots = [(0, 256), (2 ** 30 + 128, 128), (R - 64 - 128, 128 + 64)]
    for k, (r, n) in enumerate(spots):
        x[r:r + n] = workloads.normal_bf16((n, C), 1.0, 60 + k, device="cuda")
    o = fq.quantize_1x128_grouped(x, torch.tensor([0, R], dtype=torch.int32, device="cuda"))
    assert fq.device_status() == fq.FP8Q_OK
    for r, n in spots:
        few = fq.quantize_1x128_grouped(x[r:r + n], torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        tiles = -(-n // 128)
        assert torch.equal(o["q_col"][:, r:r + tiles * 128], few["q_col"][:, :tiles * 128])
        assert torch.equal(o["s_col"][r // 128:r // 128 + tiles], few["s_col"][:tiles])
    rest = o["s_col"][2:2 ** 20]
    assert bool((rest == 1).all())                                 # tiles of zeros
    del x, o, rest
    torch.cuda.empty_cache()
