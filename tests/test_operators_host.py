"""Refusals of the grouped quantizer and products, of gradient clipping and of the norms, found on the
host before anything runs (no GPU needed: a call that passed would report FP8Q_ERR_CUDA here)."""
import ctypes

import pytest
import torch

import fp4_precision_gemm_b200 as fq

P = 0x10000          # never dereferenced
VP = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    import os
    if not os.path.exists(fq.library_path):
        from fp4_precision_gemm_b200 import build
        build.build()


def passed(st):
    """A call whose arguments pass fails at the first CUDA call without a GPU."""
    return st in (fq.FP8Q_OK, fq.FP8Q_ERR_CUDA)


def test_capacity():
    assert fq.fp8q_grouped_capacity(0, 4) == 0 and fq.fp8q_grouped_capacity(5, 0) == 0
    assert fq.fp8q_grouped_capacity(-1, 4) == 0
    assert fq.fp8q_grouped_capacity(1, 256) == 128
    assert fq.fp8q_grouped_capacity(8, 32) == 8 * 128
    assert fq.fp8q_grouped_capacity(1000, 8) == 15 * 128
    for rows in (1, 7, 127, 128, 129, 4000):
        for groups in (1, 3, 64):
            cap = fq.fp8q_grouped_capacity(rows, groups) // 128
            # the worst split: one row in most experts, the rest in one
            worst = [1] * min(groups - 1, rows - 1) + [rows - min(groups - 1, rows - 1)]
            assert cap >= sum(-(-n // 128) for n in worst)


def test_grouped_quantizer_refusals():
    def call(x=P, rows=300, cols=256, ld=256, offs=P, groups=3, qr=None, sr=None, ldr=0, qc=P, sc=P, ldc=256):
        return fq.fp8q_quantize_1x128_grouped(VP(x), rows, cols, ld, VP(offs), groups, VP(qr), VP(sr), ldr, VP(qc),
                                              VP(sc), ldc, None)
    assert call(rows=0) == fq.FP8Q_OK and call(cols=0, ld=0) == fq.FP8Q_OK
    assert call(rows=-1) == fq.FP8Q_ERR_SHAPE
    assert call(groups=0) == fq.FP8Q_ERR_SHAPE and call(groups=257) == fq.FP8Q_ERR_UNSUPPORTED
    assert call(offs=None) == fq.FP8Q_ERR_NULL and call(qc=None) == fq.FP8Q_ERR_NULL and call(sc=None) == fq.FP8Q_ERR_NULL
    assert call(qr=P) == fq.FP8Q_ERR_NULL                                    # codes without scales
    assert call(cols=200, ld=200) == fq.FP8Q_ERR_SHAPE                       # colwise: cols % 16
    assert call(cols=240, ld=240, qr=P, sr=P, ldr=300) == fq.FP8Q_ERR_SHAPE  # rowwise: cols % 128
    assert call(qr=P, sr=P, ldr=296) == fq.FP8Q_ERR_SHAPE and call(ldc=252) == fq.FP8Q_ERR_SHAPE
    assert call(ldc=258) == fq.FP8Q_ERR_SHAPE and call(ld=252) == fq.FP8Q_ERR_SHAPE
    assert call(x=P + 8) == fq.FP8Q_ERR_ALIGN and call(qc=P + 8) == fq.FP8Q_ERR_ALIGN


def gemm_args(**kw):
    a = fq.GemmArgs()
    a.recipe, a.layout = fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD
    a.M, a.N, a.K = 256, 256, 512
    a.a = a.b = a.c = a.a_scale = a.b_scale = a.m_offsets = P
    a.lda = a.ldb = 512
    a.ld_sa, a.ld_sb, a.ldc, a.num_groups = 256, 256, 256, 4
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_grouped_product_refusals():
    call = lambda **kw: fq.fp8q_gemm_blockscaled(gemm_args(**kw), None)  # noqa: E731
    dgrad = dict(layout=fq.FP8Q_DGRAD, ld_sb=2)
    assert call(num_groups=257) == fq.FP8Q_ERR_UNSUPPORTED and call(num_groups=-1) == fq.FP8Q_ERR_SHAPE
    assert call(recipe=fq.FP8Q_MXFP8) == fq.FP8Q_ERR_UNSUPPORTED
    assert call(m_offsets=None) == fq.FP8Q_ERR_NULL and call(m_offsets=None, **dgrad) == fq.FP8Q_ERR_NULL
    assert call(q_out=P, s_out=P, ld_q_out=256, ld_s_out=256) == fq.FP8Q_ERR_UNSUPPORTED
    assert call(ld_sb=252) == fq.FP8Q_ERR_SHAPE and call(**{**dgrad, "ld_sb": 1}) == fq.FP8Q_ERR_SHAPE
    assert call(K=500) == fq.FP8Q_ERR_SHAPE
    # rows of the stacked C (wgrad) and B (fprop, dgrad) are 32-bit
    assert call(M=1 << 29, ld_sa=1 << 29) == fq.FP8Q_ERR_SHAPE
    assert call(N=1 << 29, ldc=1 << 29, layout=fq.FP8Q_DGRAD, ld_sb=1 << 22) == fq.FP8Q_ERR_SHAPE


def test_grouped_gemm_binding_refusals():
    """Shapes that the binding can see to be wrong; everything right but the device is refused last."""
    a, b = torch.zeros((8, 128), dtype=torch.uint8), torch.zeros((2, 128, 128), dtype=torch.uint8)
    offs = torch.tensor([0, 4, 8], dtype=torch.int32)
    sa, sb = torch.ones((1, 8)), torch.ones((2, 1, 1))
    bf16 = torch.bfloat16

    def refused(why, a=a, b=b, m_offsets=offs, a_scale=sa, b_scale=sb, **kw):
        with pytest.raises(ValueError, match=why):
            fq.gemm(a, b, m_offsets=m_offsets, a_scale=a_scale, b_scale=b_scale, **kw)

    refused("CUDA device")
    refused("CUDA device", layout=fq.FP8Q_DGRAD, out=torch.zeros((8, 128), dtype=bf16))
    refused("m_offsets", m_offsets=offs.long())
    refused("m_offsets", m_offsets=offs[::2])
    refused("m_offsets", m_offsets=offs[:1])
    refused("must be .G, N, K.", b=b[0])                                     # one matrix for two experts
    refused("one matrix per expert", b=b[:1])
    refused("one matrix per expert", b=torch.zeros((4, 128, 128), dtype=torch.uint8)[::2])
    refused("uint8", a=torch.zeros((8, 128)))
    refused("uint8", a=torch.zeros((128, 8), dtype=torch.uint8).t())
    refused("same K", a=torch.zeros((8, 256), dtype=torch.uint8), a_scale=torch.ones((2, 8)))
    for bad in (torch.ones((1, 4)), torch.ones(8), torch.ones((1, 16))[:, ::2], sa.double()):
        refused("a_scale", a_scale=bad)
    for bad in (torch.ones((1, 1, 1)), torch.ones((2, 1, 2)), torch.ones((2, 1)), sb.bfloat16()):
        refused("b_scale", b_scale=bad)
    for bad in (torch.zeros((8, 128)), torch.zeros((7, 128), dtype=bf16), torch.zeros((128, 8), dtype=bf16).t()):
        refused("`out`", out=bad)
    refused("FP32 `out`", accumulate_fp32=True)
    # wgrad: 2-D operands, scales of every chunk, a stacked result
    w = dict(a=torch.zeros((8, 256), dtype=torch.uint8), b=torch.zeros((16, 256), dtype=torch.uint8),
             layout=fq.FP8Q_WGRAD, a_scale=torch.ones((2, 8)), b_scale=torch.ones((2, 16)))
    refused("CUDA device", **w)
    refused("padded token axis", layout=fq.FP8Q_WGRAD)
    refused("a_scale", **{**w, "a_scale": torch.ones((1, 8))})
    refused("b_scale", **{**w, "b_scale": torch.ones((1, 16))})
    refused("`out`", **w, out=torch.zeros((2, 8, 64)), accumulate_fp32=True)
    refused("`out`", **w, out=torch.zeros((4, 8, 16))[::2], accumulate_fp32=True)


def items(*rows):
    return (fq.GradItem * max(1, len(rows)))(*[fq.GradItem(*r) for r in rows])


def clip(rows, max_norm=1.0, eps=1e-6, norm=P, ws=P, nbytes=1 << 20):
    return fq.fp8q_clip_grad_norm(items(*rows), len(rows), max_norm, eps, VP(norm), VP(ws), nbytes, None)


def test_clip_refusals():
    ok = (P, P, 100, fq.FP8Q_FP32)
    assert passed(clip([ok])) and passed(clip([])) and passed(clip([ok], norm=None))
    assert passed(clip([(None, None, 0, fq.FP8Q_BF16)]))
    assert fq.fp8q_clip_grad_norm(None, 1, 1.0, 0.0, None, VP(P), 1 << 20, None) == fq.FP8Q_ERR_NULL
    assert fq.fp8q_clip_grad_norm(None, -1, 1.0, 0.0, None, VP(P), 1 << 20, None) == fq.FP8Q_ERR_SHAPE
    assert clip([(P, P, 100, 2)]) == fq.FP8Q_ERR_UNSUPPORTED
    assert clip([(P, P, -1, 0)]) == fq.FP8Q_ERR_SHAPE
    assert clip([(None, P, 1, 0)]) == fq.FP8Q_ERR_NULL and clip([(P, None, 1, 0)]) == fq.FP8Q_ERR_NULL
    assert clip([(P + 2, P, 1, fq.FP8Q_FP32)]) == fq.FP8Q_ERR_ALIGN
    assert clip([(P + 1, P, 1, fq.FP8Q_BF16)]) == fq.FP8Q_ERR_ALIGN
    for bad in (-1.0, float("nan")):
        assert clip([ok], max_norm=bad) == fq.FP8Q_ERR_SHAPE
    for bad in (-1.0, float("nan"), float("inf")):
        assert clip([ok], eps=bad) == fq.FP8Q_ERR_SHAPE
    assert clip([ok], ws=None) == fq.FP8Q_ERR_NULL and clip([ok], ws=P + 8) == fq.FP8Q_ERR_ALIGN
    need = fq.fp8q_clip_grad_workspace_bytes(1)
    assert clip([ok], nbytes=need - 1) == fq.FP8Q_ERR_SHAPE and passed(clip([ok], nbytes=need))
    assert fq.fp8q_clip_grad_workspace_bytes(1025) == 2 * need and fq.fp8q_clip_grad_workspace_bytes(-1) == 0
    assert fq.fp8q_clip_grad_workspace_bytes(0) == need


def test_clip_overlaps():
    f = fq.FP8Q_FP32
    bad = fq.FP8Q_ERR_UNSUPPORTED
    assert clip([(P, P, 100, f), (P, P, 100, f)]) == bad                       # one gradient twice, in place
    assert clip([(P, P, 100, f), (P + 396, P + 396, 100, f)]) == bad           # overlapping by one element
    assert passed(clip([(P, P, 100, f), (P + 400, P + 400, 100, f)]))
    assert clip([(P, P + 4, 100, f)]) == bad                                   # out shifted over its own grad
    assert clip([(P, P + 4000, 100, f), (P + 4200, P + 8000, 100, f)]) == bad  # out over another's grad
    assert passed(clip([(P, P + 4000, 100, f), (P, P + 8000, 100, f)]))        # one gradient, two copies
    assert clip([(P, P, 100, f), (P, P + 8000, 100, f)]) == bad                # one of them in place
    assert clip([(P, P + 4000, 100, f), (P + 8000, P + 4200, 10, f)]) == bad   # outs overlap
    assert clip([(P, P, 100, f), (P + 100, P + 9000, 0, f), (P + 396, P + 9000, 3, fq.FP8Q_BF16)]) == bad


def test_clip_binding_refusals():
    with pytest.raises(ValueError):
        fq.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        fq.clip_grad_norm([torch.zeros(4)], 1.0)                               # not on a GPU
    with pytest.raises(ValueError):
        fq.clip_grad_norm([torch.zeros(4)], 1.0, out=[])


def norm_args(cls, **kw):
    a = cls()
    a.rows, a.cols, a.alpha = 4, 256, 1.0
    for f, t in cls._fields_:
        if f.startswith("ld_"):
            setattr(a, f, 256)
        elif t is ctypes.c_void_p:
            setattr(a, f, P)
    if cls is fq.NormBackwardArgs:
        a.workspace_bytes = 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_norm_refusals():
    call = lambda **kw: fq.fp8q_norm_residual(norm_args(fq.NormArgs, **kw), None)  # noqa: E731
    assert fq.lib().fp8q_norm_residual(None, None) == fq.FP8Q_ERR_NULL
    assert call(rows=0) == fq.FP8Q_OK and call(rows=0, y=None, h=None) == fq.FP8Q_OK
    if not torch.cuda.is_available():
        assert call() == fq.FP8Q_ERR_CUDA and call(w_post=None, gate=None, rstd_pre=None, rstd_post=None) == fq.FP8Q_ERR_CUDA
        assert call(n_out=None) == fq.FP8Q_ERR_CUDA and call(q_row=None, s_row=None) == fq.FP8Q_ERR_CUDA
    assert call(h_dtype=2) == fq.FP8Q_ERR_UNSUPPORTED and call(w_dtype=-1) == fq.FP8Q_ERR_UNSUPPORTED
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=252), dict(cols=16392), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(ld_y=248), dict(ld_h=260), dict(ld_h_out=255), dict(ld_n=8), dict(cols=200),
                dict(ld_s_row=3), dict(ld_s_row=6)):
        assert call(**bad) == fq.FP8Q_ERR_SHAPE, bad
    for f in ("y", "h", "h_out", "w_pre", "q_row", "s_row"):
        assert call(**{f: None}) == fq.FP8Q_ERR_NULL, f
    assert call(n_out=None, q_row=None, s_row=None) == fq.FP8Q_ERR_NULL
    for f in ("y", "h", "h_out", "w_pre", "w_post", "gate", "n_out", "q_row"):
        assert call(**{f: P + 8}) == fq.FP8Q_ERR_ALIGN, f


def test_norm_backward_refusals():
    call = lambda **kw: fq.fp8q_norm_residual_backward(norm_args(fq.NormBackwardArgs, **kw), None)  # noqa: E731
    assert fq.lib().fp8q_norm_residual_backward(None, None) == fq.FP8Q_ERR_NULL
    if not torch.cuda.is_available():
        assert call() == fq.FP8Q_ERR_CUDA
        assert call(w_post=None, rstd_post=None, gate=None, dw_post=None, dgate=None) == fq.FP8Q_ERR_CUDA
        assert fq.fp8q_norm_backward_workspace_bytes(4, 256, 0) == 0
    assert call(h_dtype=2) == fq.FP8Q_ERR_UNSUPPORTED and call(w_dtype=7) == fq.FP8Q_ERR_UNSUPPORTED
    for bad in (dict(rows=-1), dict(cols=4), dict(cols=20000), dict(ld_dn=255), dict(ld_dh_out=248), dict(ld_y=0),
                dict(ld_h=252), dict(ld_dh=-8), dict(ld_dy=8)):
        assert call(**bad) == fq.FP8Q_ERR_SHAPE, bad
    for f in ("dn", "dh_out", "y", "h", "w_pre", "rstd_pre", "rstd_post", "dh", "dy", "dw_pre", "workspace"):
        assert call(**{f: None}) == fq.FP8Q_ERR_NULL, f
    assert call(w_post=None, rstd_post=None) == fq.FP8Q_ERR_NULL             # dw_post without w_post
    assert call(gate=None) == fq.FP8Q_ERR_NULL                               # dgate without gate
    for f in ("dn", "dh_out", "y", "h", "w_pre", "w_post", "gate", "dh", "dy", "workspace"):
        assert call(**{f: P + 8}) == fq.FP8Q_ERR_ALIGN, f
    assert fq.fp8q_norm_backward_workspace_bytes(4, 100, 0) == 0 == fq.fp8q_norm_backward_workspace_bytes(4, 256, 2)


def test_norm_binding_refusals():
    y = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fq.norm_residual(y, y, y[0])                                         # not on a GPU
    with pytest.raises(ValueError):
        fq.norm_residual_backward(y, y, y, y, torch.ones(4), y[0], w_post=y[0])


@pytest.mark.skipif(__import__("shutil").which("gcc") is None, reason="needs gcc")
def test_binding_structs_match_the_header(tmp_path):
    """Sizes and offsets of the ctypes mirrors against a C compiler's."""
    import os
    import subprocess
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    mirrors = {"fp8q_grad_item": fq.GradItem, "fp8q_norm_args": fq.NormArgs, "fp8q_norm_backward_args": fq.NormBackwardArgs}
    lines = []
    for cname, cls in mirrors.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, *_ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "fp8q.h"\nint main(void) {' + "\n".join(lines) + "return 0;}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", header, "-o", exe, str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([exe], check=True, capture_output=True,
                                                       text=True).stdout.splitlines())
    for cname, cls in mirrors.items():
        assert int(got[cname]) == ctypes.sizeof(cls)
        for f, *_ in cls._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(cls, f).offset, (cname, f)
