"""Clipping by factors below FP32's normal range (a norm of 1e38 times the limit and more).

Tolerances: the norm of one size's values is off by at most 5 * 2^-24 of itself before it is rounded to FP32
(eight squares added in FP32, the rest in FP64), so is the factor; the product is rounded to FP32 once, and for
BF16 once more: 7 * 2^-24, and 2^-8 of the value.  Clipped values are in the normal range of both types here."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16
VALUE = {F: 7 * 2.0 ** -24, B: 7 * 2.0 ** -24 + 2.0 ** -8}


@pytest.mark.parametrize("place", ["in place", "out"])
@pytest.mark.parametrize("max_norm", [1.0, 3.0, 1e-8, 1e-30])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("n", [1, 7, 10007])
def test_factors_below_the_normal_range(cuda_lib, n, dtype, max_norm, place):
    g = torch.Generator(device="cuda").manual_seed(n)
    t = ((torch.rand(n, generator=g, device="cuda") + 1.0) * 1.5e38).to(dtype)
    t[::2] *= -1.0
    before = t.double()
    norm = math.sqrt(math.fsum((before ** 2).tolist()))
    out = t if place == "in place" else torch.empty_like(t)
    cuda_lib.clip_grad_norm([t], max_norm, out=None if place == "in place" else [out])
    want = before * (max_norm / (norm + 1e-6))
    assert float(want.abs().min()) > torch.finfo(dtype).tiny
    assert bool(((out.double() - want).abs() <= VALUE[dtype] * want.abs()).all())
    if place == "out":
        assert torch.equal(t.double(), before)


@pytest.mark.parametrize("dtype", [F, B])
def test_small_values_beside_them(cuda_lib, dtype):
    """The clipped copy of a small value is rounded to what its type has: half a step of the subnormals."""
    t = torch.tensor([3e38, -3e38, 1e10, 1.0, 0.0, -0.0, 1e-30, -2e30], device="cuda").to(dtype)
    before = t.double()
    norm = math.sqrt(math.fsum((before ** 2).tolist()))
    cuda_lib.clip_grad_norm([t], 0.5)
    want = before * (0.5 / (norm + 1e-6))
    step = 2.0 ** -149 if dtype == F else 2.0 ** -133
    assert bool(((t.double() - want).abs() <= VALUE[dtype] * want.abs() + step).all())
    assert bool(torch.equal(torch.signbit(t), torch.signbit(before)))
