"""What the grouped gemm() of the binding refuses and takes, found on the host (no GPU needed: a call with nothing
else wrong is refused for its host tensors, last of all)."""
import pytest
import torch

import fp4_precision_gemm_b200 as fq

U8, F32, BF16 = torch.uint8, torch.float32, torch.bfloat16
LAST = "must be on a CUDA device"


def operands(layout, M=8, K=256, N=256, G=2):
    """a, b, a_scale, b_scale of the smallest shapes, and the offsets."""
    o = dict(m_offsets=torch.tensor([0] + [M] * G, dtype=torch.int32), layout=layout, a=torch.zeros((M, K), dtype=U8),
             a_scale=torch.ones((K // 128, M)))
    if layout == fq.FP8Q_WGRAD:
        return {**o, "b": torch.zeros((N, K), dtype=U8), "b_scale": torch.ones((K // 128, N))}
    kb, nb = K // 128, -(-N // 128)
    return {**o, "b": torch.zeros((G, N, K), dtype=U8),
            "b_scale": torch.ones((G, nb, kb) if layout == fq.FP8Q_FPROP else (G, kb, nb))}


def refused(why, **kw):
    with pytest.raises(ValueError, match=why):
        fq.gemm(**kw)


LAYOUTS = [fq.FP8Q_FPROP, fq.FP8Q_DGRAD, fq.FP8Q_WGRAD]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_an_explicit_k_stays_within_the_operands(layout):
    """K up to the row stride of a slice passes the strides' checks further down: scales and codes of columns that
    the slice does not have would be read."""
    o = operands(layout)
    refused(LAST, **o)
    refused(LAST, **o, K=256)
    half = {**o, "b_scale": operands(layout, K=128)["b_scale"]}
    refused(LAST, **half, K=128)                                  # fewer columns than there are
    refused("K must", **o, K=384)
    refused("K must", **o, K=-128)
    wide_a, wide_b = {**o, "a": torch.zeros((8, 512), dtype=U8)[:, :256]}, o["b"].new_zeros((*o["b"].shape[:-1], 512))
    refused(LAST, **wide_a)
    refused("K must", **wide_a, K=512)
    refused("K must", **{**o, "a": torch.zeros((8, 512), dtype=U8), "b": wide_b[..., :256]}, K=512)
    # scales are compared with the K that is meant
    refused(LAST, **{**half, "a_scale": o["a_scale"][:1]}, K=128)
    refused("a_scale must", **{**o, "a_scale": o["a_scale"][:1]})


@pytest.mark.parametrize("layout", LAYOUTS)
def test_explicit_leading_dimensions_stay_within_the_scales(layout):
    o = operands(layout)
    a, b = o["a_scale"], o["b_scale"]
    rows, cols = (2, 256) if layout == fq.FP8Q_WGRAD else (4, 2)
    refused(LAST, **o, ld_sa=8)
    refused(LAST, **o, ld_sb=cols)
    refused("a_scale must", **o, ld_sa=12)                        # the last row would end past the tensor
    refused("a_scale must", **o, ld_sa=4)                         # rows over one another
    refused("a_scale must", **{**o, "a_scale": a[:1]}, ld_sa=8)
    refused("a_scale must", **{**o, "a_scale": a.double()}, ld_sa=8)
    refused("b_scale must", **o, ld_sb=cols + 4)
    refused("b_scale must", **o, ld_sb=cols - 1)
    refused("b_scale must", **{**o, "b_scale": b[:1]}, ld_sb=cols)
    refused("b_scale must", **{**o, "b_scale": b.double()}, ld_sb=cols)
    # slices of wider buffers, and flat ones
    refused(LAST, **{**o, "a_scale": torch.ones((2, 20))[:, 4:12]}, ld_sa=20)
    refused("a_scale must", **{**o, "a_scale": torch.ones((2, 20))[:, 4:11]}, ld_sa=20)
    refused(LAST, **{**o, "a_scale": torch.ones(16)}, ld_sa=8)
    refused("a_scale must", **{**o, "a_scale": torch.ones(15)}, ld_sa=8)
    refused(LAST, **{**o, "b_scale": torch.ones((rows, cols + 4))[:, :cols]}, ld_sb=cols + 4)
    refused("b_scale must", **{**o, "b_scale": torch.ones((rows, cols + 4))[:, :cols - 1]}, ld_sb=cols + 4)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_what_is_read_counts_and_not_its_spelling(layout):
    """Calls whose tensors hold all that the kernels read, where they read it: nothing but the device is wrong."""
    o = operands(layout)
    wgrad = layout == fq.FP8Q_WGRAD
    for t in (torch.float8_e4m3fn, torch.int8):
        refused(LAST, **{**o, "a": o["a"].view(t), "b": o["b"].view(t)})
    refused(LAST, **{**o, "b": torch.zeros((*o["b"].shape[:-1], 384), dtype=U8)})         # more columns than a
    refused(LAST, **{**o, "m_offsets": o["m_offsets"][None]})
    refused(LAST, **{**o, "a_scale": torch.ones((3, 20))})                                # rows and columns to spare
    if wgrad:
        refused(LAST, **{**o, "b_scale": torch.ones((3, 260))})
        return
    G, r, c = o["b_scale"].shape
    refused(LAST, **{**o, "b_scale": torch.ones((G * r, c))})                             # the experts' rows stacked
    refused(LAST, **{**o, "b_scale": torch.ones((1, G * r, c))})
    refused(LAST, **{**o, "b_scale": torch.ones((G, r, c + 2))})
    refused(LAST, **{**o, "b_scale": torch.ones((G * r, c + 2))})
    refused(LAST, **{**o, "b_scale": torch.ones((G + 1, r, c)), "b": torch.zeros((G + 1, 256, 256), dtype=U8)})
    refused(LAST, **o, out=torch.zeros((11, 256), dtype=BF16))
    refused(LAST, **o, out=torch.zeros((8, 264), dtype=BF16))
    refused(LAST, **o, out=torch.zeros((11, 264)), accumulate_fp32=True)
    one = operands(layout, G=1)                                    # one expert: the distance to a second means nothing
    refused(LAST, **{**one, "b": torch.zeros((3, 256, 256), dtype=U8)[::2][:1]})


@pytest.mark.parametrize("layout", LAYOUTS)
def test_what_is_read_and_not_there_is_refused(layout):
    o = operands(layout)
    wgrad = layout == fq.FP8Q_WGRAD
    for t in (torch.float8_e5m2, torch.bfloat16, torch.bool):
        refused("codes", **{**o, "a": torch.zeros((8, 256), dtype=t)})
    refused("same K", **{**o, "b": torch.zeros((*o["b"].shape[:-1], 128), dtype=U8)})
    refused("a_scale must", **{**o, "a_scale": torch.ones((2, 7))})
    refused("a_scale must", **{**o, "a_scale": torch.ones((1, 16))})
    refused("a_scale must", **{**o, "a_scale": torch.ones((2, 16))[:, :8]})               # its row stride is not given
    refused("`out`", **o, out=torch.zeros((2, 7, 256) if wgrad else (7, 256), dtype=BF16))
    refused("`out`", **o, out=torch.zeros((2, 8, 255) if wgrad else (8, 255), dtype=BF16))
    refused("`out`", **o, out=torch.zeros((2, 8, 256) if wgrad else (8, 256)))
    if wgrad:
        refused("b_scale must", **{**o, "b_scale": torch.ones((2, 255))})
        refused("`out`", **o, out=torch.zeros((2, 9, 256), dtype=BF16))
        return
    G, r, c = o["b_scale"].shape
    refused("b_scale must", **{**o, "b_scale": torch.ones((G, r + 1, c))})                # experts too far apart
    refused("b_scale must", **{**o, "b_scale": torch.ones((G, r - 1, c))})
    refused("b_scale must", **{**o, "b_scale": torch.ones((G * r - 1, c))})
    refused("b_scale must", **{**o, "b_scale": torch.ones((G, r, c - 1))})
    refused("b_scale must", **{**o, "b_scale": torch.ones((G - 1, r, c))})
    refused("b_scale must", **{**o, "b_scale": torch.ones((G * r * c,))})
    refused("one matrix per expert", **{**o, "b": o["b"][:1]})
    refused("one matrix per expert", **{**o, "b": torch.zeros((4, 256, 256), dtype=U8)[::2]})
