"""Products grouped by expert in every direction and the grouped 1x128 quantizer.

References are in 64 bits from the codes and scales that the kernel is given.  Tolerance of a
product, elementwise, with T = |A_dq| |B_dq|^T: within a chunk the tensor core adds 128 products
in some order, each addition off by at most one unit in the last place (2^-23) of the sum of
magnitudes; a chunk's promotion rounds its scale product, its multiplication and its addition
(2^-24 each, at most once per chunk for the running sum), so
    |sum - ref| <= (128 * 2^-23 + (K/128 + 3) * 2^-24) T =: gamma T,
a BF16 C adds half a step, 2^-8 (|ref| + gamma T), and FP32 accumulation one more addition,
2^-24 (|C_before| + |ref| + gamma T)."""
import numpy as np
import pytest
import torch

import workloads
from oracle import quant as Q

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def gamma(chunks):
    return 128 * 2.0 ** -23 + (chunks + 3) * 2.0 ** -24


def codes(shape, seed):
    """Random E4M3 codes (no NaN) on the device."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).mul_(60.0).clamp_(-448, 448).to(E4M3).view(torch.uint8).cuda()


def scales(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.exp2(torch.randn(shape, generator=g)).mul_(0.01).cuda()


def values(q):
    return q.view(E4M3).double()


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def rows_reference(a, sa, b, sb, counts, dgrad):
    """C and T (64 bits): rows of expert e times its matrix."""
    M, K = a.shape
    x = values(a) * sa[:, :M].double().t().repeat_interleave(128, 1)
    c, t, at = [], [], 0
    for e, n in enumerate(counts):
        blocks = (sb[e].t() if dgrad else sb[e]).double()
        w = values(b[e]) * blocks.repeat_interleave(128, 0)[:b.shape[1]].repeat_interleave(128, 1)
        xe = x[at:at + n]
        c.append(xe @ w.t())
        t.append(xe.abs() @ w.abs().t())
        at += n
    return torch.cat(c), torch.cat(t)


def assert_within(got, ref, bound, what):
    over = (got.double() - ref).abs() - bound
    assert torch.isfinite(got.double()).all(), what
    assert float(over.max()) <= 0, f"{what}: worst {float(over.max())} over the bound"


COUNTS = [
    [130, 0, 1, 257, 60, 128],
    [0, 0, 5],
    [1],
    [1] * 40 + [0] * 20 + [3],
    [700, 2, 0, 31],
    [17] * 256,
]


@pytest.mark.parametrize("layout", ["fprop", "dgrad"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("K,N", [(384, 256), (1152, 200), (128, 8)])
def test_rows(cuda_lib, layout, counts, K, N):
    """Ragged experts, empty ones among them; N that ends inside a tile; a last scale block cut by N."""
    fq = cuda_lib
    G, M, nb = len(counts), sum(counts), -(-N // 128)
    dgrad = layout == "dgrad"
    a, b = codes((M, K), 1), codes((G, N, K), 2)
    sa, sb = scales((K // 128, M + -M % 4), 3), scales((G, K // 128, nb) if dgrad else (G, nb, K // 128), 4)
    lay = fq.FP8Q_DGRAD if dgrad else fq.FP8Q_FPROP
    ref, t = rows_reference(a, sa, b, sb, counts, dgrad)
    ga = gamma(K // 128)
    guard = torch.full((M + 300, N), 7.0, dtype=torch.bfloat16, device="cuda")
    c = fq.gemm(a, b, fq.FP8Q_BLOCKWISE, lay, a_scale=sa, b_scale=sb, m_offsets=offsets(counts), out=guard[:M])
    assert fq.device_status() == fq.FP8Q_OK
    assert_within(c, ref, ga * t + 2.0 ** -8 * (ref.abs() + ga * t), "bf16")
    assert bool((guard[M:] == 7.0).all())                 # rows behind the last expert's stay as they were
    acc = torch.randn((M, N), device="cuda")
    before = acc.double()
    fq.gemm(a, b, fq.FP8Q_BLOCKWISE, lay, a_scale=sa, b_scale=sb, m_offsets=offsets(counts), out=acc,
            accumulate_fp32=True)
    assert_within(acc, ref + before, ga * t + 2.0 ** -24 * (before.abs() + ref.abs() + ga * t), "fp32 accumulate")


@pytest.mark.parametrize("layout", ["fprop", "dgrad"])
def test_rows_padded_strides_and_stream(cuda_lib, layout):
    """Row strides wider than the matrices, outputs inside a wider buffer, on a stream of its own."""
    fq = cuda_lib
    counts, K, N = [100, 0, 33, 300], 256, 264
    G, M, nb = len(counts), sum(counts), 3
    dgrad = layout == "dgrad"
    a = torch.empty((M, K + 32), dtype=torch.uint8, device="cuda")[:, :K]
    b = torch.empty((G, N, K + 16), dtype=torch.uint8, device="cuda")[:, :, :K]
    a.copy_(codes((M, K), 11))
    b.copy_(codes((G, N, K), 12))
    sa, sb = scales((K // 128, M + 8), 13), scales((G, K // 128, nb) if dgrad else (G, nb, K // 128), 14)
    wide = torch.full((M, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    offs = offsets(counts)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    fq.gemm(a, b, fq.FP8Q_BLOCKWISE, fq.FP8Q_DGRAD if dgrad else fq.FP8Q_FPROP, a_scale=sa, b_scale=sb, m_offsets=offs,
            out=wide[:, :N], stream=st)
    st.synchronize()
    ref, t = rows_reference(a.contiguous(), sa, b.contiguous(), sb, counts, dgrad)
    ga = gamma(K // 128)
    assert_within(wide[:, :N], ref, ga * t + 2.0 ** -8 * (ref.abs() + ga * t), "strided")
    assert bool((wide[:, N:] == 7.0).all())


@pytest.mark.parametrize("layout", ["fprop", "dgrad"])
@pytest.mark.parametrize("counts", [[1], [0, 7, 0, 33, 64, 1], [512], [3] * 100, [100, 0, 412]], ids=str)
def test_few_rows_equal_many_rows_to_the_bit(cuda_lib, layout, counts):
    """The same rows alone, and in front of another expert's thousand rows: whatever kernel a size
    selects, a row's result is the same sum in the same order."""
    fq = cuda_lib
    G, M, K, N, extra = len(counts), sum(counts), 640, 392, 1000
    dgrad = layout == "dgrad"
    a, b = codes((M + extra, K), 71), codes((G + 1, N, K), 72)
    sa, sb = scales((K // 128, M + extra), 73), scales((G + 1, 5, 4) if dgrad else (G + 1, 4, 5), 74)
    lay = fq.FP8Q_DGRAD if dgrad else fq.FP8Q_FPROP
    acc = torch.randn((M + extra, N), device="cuda")
    few, many = acc[:M].clone(), acc.clone()
    for out in (None, 1):
        one = fq.gemm(a[:M], b[:G], layout=lay, a_scale=sa, b_scale=sb[:G], m_offsets=offsets(counts),
                      out=few if out else None, accumulate_fp32=bool(out))
        all_ = fq.gemm(a, b, layout=lay, a_scale=sa, b_scale=sb, m_offsets=offsets(counts + [extra]),
                       out=many if out else None, accumulate_fp32=bool(out))
        assert torch.equal(one, all_[:M])


@pytest.mark.parametrize("extra", [0, 1500])
@pytest.mark.parametrize("layout", ["fprop", "dgrad"])
def test_rows_of_other_experts_do_not_leak(cuda_lib, layout, extra):
    """NaN codes and scales in one expert's rows and matrix leave the others' results alone (in the kernel for few
    rows and, with many more behind them, in the other)."""
    fq = cuda_lib
    counts, K, N = [37, 20, 100 + extra], 256, 144
    G, M = 3, sum(counts)
    dgrad = layout == "dgrad"
    a, b = codes((M, K), 81), codes((G, N, K), 82)
    sa, sb = scales((2, M + -M % 4), 83), scales((G, 2, 2), 84)
    call = lambda: fq.gemm(a, b, layout=fq.FP8Q_DGRAD if dgrad else fq.FP8Q_FPROP, a_scale=sa, b_scale=sb,  # noqa: E731
                           m_offsets=offsets(counts))
    clean = call()
    a[37:57] = 0x7F
    b[1] = 0x7F
    sa[:, 37:57] = float("nan")
    sb[1] = float("inf")
    got = call()
    assert torch.equal(got[:37], clean[:37]) and torch.equal(got[57:], clean[57:])
    assert bool(got[37:57].isnan().all())


@pytest.mark.parametrize("layout", ["fprop", "dgrad"])
@pytest.mark.parametrize("offs", [[0, 700, 300, 2000], [0, 700, 9000, 2000], [-3, 700, 900, 2000]])
def test_many_rows_offsets_out_of_rule(cuda_lib, layout, offs):
    fq = cuda_lib
    M, K, N, G = 2000, 256, 144, 3
    dgrad = layout == "dgrad"
    a, b, sa, sb = codes((M, K), 91), codes((G, N, K), 92), scales((2, M), 93), scales((G, 2, 2), 94)
    guard = torch.full((M + 300, N), 7.0, dtype=torch.bfloat16, device="cuda")
    assert fq.device_status() == fq.FP8Q_OK
    fq.gemm(a, b, layout=fq.FP8Q_DGRAD if dgrad else fq.FP8Q_FPROP, a_scale=sa, b_scale=sb,
            m_offsets=torch.tensor(offs, dtype=torch.int32, device="cuda"), out=guard[:M])
    assert fq.device_status() == fq.FP8Q_ERR_DEVICE_ARG
    assert bool((guard[M:] == 7.0).all())
    clamped = [0]
    for v in offs[1:]:
        clamped.append(min(max(v, clamped[-1]), M))
    counts = [q - p for p, q in zip(clamped, clamped[1:])]
    n = sum(counts)
    ref, t = rows_reference(a[:n], sa, b, sb, counts, dgrad)
    assert_within(guard[:n], ref, gamma(2) * t + 2.0 ** -8 * (ref.abs() + gamma(2) * t), "clamped")


def wgrad_reference(x, sx, y, sy, counts):
    c, t, at = [], [], 0
    for n in counts:
        k = -(-n // 128)
        xe, ye = (values(q[:, at * 128:(at + k) * 128].contiguous())
                  * s[at:at + k, :q.shape[0]].double().t().repeat_interleave(128, 1) for q, s in ((x, sx), (y, sy)))
        c.append(xe @ ye.t())
        t.append(xe.abs() @ ye.abs().t())
        at += k
    return torch.stack(c), torch.stack(t)


@pytest.mark.parametrize("counts", COUNTS[:5], ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("M,N", [(256, 256), (208, 528), (16, 16), (1040, 48)])
def test_wgrad(cuda_lib, counts, M, N):
    """dW_e over each expert's own tokens: BF16 (zeros for an expert without tokens) and FP32
    accumulation (its C unchanged, to the bit), M and N that end inside a tile."""
    fq = cuda_lib
    G, R = len(counts), sum(counts)
    P = fq.fp8q_grouped_capacity(R, G)
    assert P >= sum(-(-n // 128) for n in counts) * 128
    x, y = codes((M, P), 21), codes((N, P), 22)
    sx, sy = scales((P // 128, M + -M % 4), 23), scales((P // 128, N + -N % 4), 24)
    offs = offsets(counts)
    ref, t = wgrad_reference(x, sx, y, sy, counts)
    ga = gamma(-(-max(counts) // 128))
    c = fq.gemm(x, y, fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD, a_scale=sx, b_scale=sy, m_offsets=offs)
    assert c.shape == (G, M, N) and c.dtype == torch.bfloat16
    assert_within(c, ref, ga * t + 2.0 ** -8 * (ref.abs() + ga * t), "bf16")
    acc = torch.randn((G, M, N), device="cuda")
    acc[0, 0, 0] = -0.0
    before = acc.clone()
    fq.gemm(x, y, fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD, a_scale=sx, b_scale=sy, m_offsets=offs, out=acc,
            accumulate_fp32=True)
    assert fq.device_status() == fq.FP8Q_OK
    b64 = before.double()
    assert_within(acc, ref + b64, ga * t + 2.0 ** -24 * (b64.abs() + ref.abs() + ga * t), "fp32 accumulate")
    for e, n in enumerate(counts):
        if n == 0:
            assert torch.equal(acc[e].view(torch.int32), before[e].view(torch.int32))
            assert bool((c[e] == 0).all())
    # the same sums every time
    again = before.clone()
    fq.gemm(x, y, fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD, a_scale=sx, b_scale=sy, m_offsets=offs, out=again,
            accumulate_fp32=True)
    assert torch.equal(acc, again)


def test_wgrad_one_group_matches_the_ungrouped_product(cuda_lib):
    """One expert with a multiple of 128 tokens is the plain WGRAD, to the bit."""
    fq = cuda_lib
    T, M, N = 512, 272, 400
    x, y, sx, sy = codes((M, T), 31), codes((N, T), 32), scales((T // 128, M), 33), scales((T // 128, N), 34)
    P = fq.fp8q_grouped_capacity(T, 1)
    pad = lambda q: torch.nn.functional.pad(q, (0, P - T), value=0x7E)  # noqa: E731 - codes of 448, not to be read
    one = torch.ones
    xp, yp = pad(x), pad(y)
    sxp = torch.cat((sx, one((P // 128 - T // 128, M), device="cuda")))
    syp = torch.cat((sy, one((P // 128 - T // 128, N), device="cuda")))
    c = fq.gemm(xp, yp, fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD, a_scale=sxp, b_scale=syp, m_offsets=offsets([T]))
    plain = fq.gemm(x, y, fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD, a_scale=sx, b_scale=sy, split_tail=False)
    assert torch.equal(c[0], plain)


@pytest.mark.parametrize("offs", [[0, 200, 100, 300], [0, 100, 100000, 300], [3, 100, 200, 300], [0, -5, 200, 300]])
def test_wgrad_offsets_out_of_rule(cuda_lib, offs):
    """Offsets that break their rule read no chunk outside the operands and are recorded."""
    fq = cuda_lib
    G, R, M, N = 3, 300, 64, 64
    P = fq.fp8q_grouped_capacity(R, G)
    x, y, sx, sy = codes((M, P), 41), codes((N, P), 42), scales((P // 128, M), 43), scales((P // 128, N), 44)
    assert fq.device_status() == fq.FP8Q_OK
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    c = fq.gemm(x, y, fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD, a_scale=sx, b_scale=sy, m_offsets=o)
    assert fq.device_status() == fq.FP8Q_ERR_DEVICE_ARG
    assert torch.isfinite(c.float()).all()


def test_no_tokens(cuda_lib):
    """No token at all: BF16 zeros, accumulators and rows as they were."""
    fq = cuda_lib
    G, M, N = 3, 48, 64
    offs = offsets([0, 0, 0])
    x = torch.zeros((0, M), dtype=torch.bfloat16, device="cuda")
    q = fq.quantize_1x128_grouped(x, offs)
    assert q["q_col"].shape == (M, 0) and q["s_col"].shape[0] == 0
    y = torch.zeros((N, 0), dtype=torch.uint8, device="cuda")
    sy = torch.zeros((0, N), device="cuda")
    c = fq.gemm(q["q_col"], y, layout=fq.FP8Q_WGRAD, a_scale=q["s_col"], b_scale=sy, m_offsets=offs)
    assert c.shape == (G, M, N) and bool((c == 0).all())
    acc = torch.randn((G, M, N), device="cuda")
    before = acc.clone()
    fq.gemm(q["q_col"], y, layout=fq.FP8Q_WGRAD, a_scale=q["s_col"], b_scale=sy, m_offsets=offs, out=acc,
            accumulate_fp32=True)
    assert torch.equal(acc, before)
    b, sb = codes((G, 64, 128), 1), scales((G, 1, 1), 2)
    r = fq.gemm(torch.zeros((0, 128), dtype=torch.uint8, device="cuda"), b, layout=fq.FP8Q_DGRAD,
                a_scale=torch.zeros((1, 4), device="cuda"), b_scale=sb, m_offsets=offs)
    assert r.shape == (0, 64)


def test_wgrad_result_past_32_bits(cuda_lib):
    """C of more than 2^31 elements: its last expert's corner, and its neighbours untouched."""
    fq = cuda_lib
    counts, M, N = [128, 0, 200], 24576, 32768          # 3 x 24576 x 32768 = 2.4e9
    P = fq.fp8q_grouped_capacity(sum(counts), 3)
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda w: torch.randn((w, P), generator=g, device="cuda").mul_(60).clamp_(-448, 448).to(E4M3).view(torch.uint8)  # noqa: E731
    x, y = rnd(M), rnd(N)
    sx, sy = (torch.rand((P // 128, w), generator=g, device="cuda") * 0.01 + 1e-3 for w in (M, N))
    c = fq.gemm(x, y, layout=fq.FP8Q_WGRAD, a_scale=sx, b_scale=sy, m_offsets=offsets(counts))
    assert fq.device_status() == fq.FP8Q_OK
    rows, cols = slice(M - 300, M), slice(N - 300, N)
    ref, t = wgrad_reference(x[rows], sx[:, rows], y[cols], sy[:, cols], counts)
    assert_within(c[:, rows, cols], ref, gamma(2) * t + 2.0 ** -8 * (ref.abs() + gamma(2) * t), "far corner")
    assert bool((c[1] == 0).all())


# ------------------------------------------------------------------------------ quantizer
def padded_oracle(bits, counts, P):
    """The oracle's colwise 1x128 of every expert's rows, zero rows appended to whole tiles."""
    C = bits.shape[1]
    q = np.zeros((C, P), np.uint8)
    s = np.ones((P // 128, C), np.float32)
    r = at = 0
    for n in counts:
        k = -(-n // 128)
        if k:
            z = np.zeros((k * 128, C), bits.dtype)
            z[:n] = bits[r:r + n]
            q[:, at * 128:(at + k) * 128], s[at:at + k] = Q.quantize_1x128_colwise(z)
        r, at = r + n, at + k
    return q, s


@pytest.mark.parametrize("rowwise", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("C", [128, 640])
def test_quantize_grouped(cuda_lib, counts, C, rowwise):
    fq = cuda_lib
    R, G = sum(counts), len(counts)
    x = workloads.normal_bf16((R, C), 1.0, 51, 1e-3, 50.0)
    x[R // 2] = 0.0
    wide = torch.full((R, C + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :C] = x.cuda()
    P = fq.fp8q_grouped_capacity(R, G)
    o = fq.quantize_1x128_grouped(wide[:, :C], offsets(counts), rowwise=rowwise)
    assert fq.device_status() == fq.FP8Q_OK
    bits = workloads.bf16_bits(x)
    q, s = padded_oracle(bits, counts, P)
    assert np.array_equal(o["q_col"].cpu().numpy(), q)
    assert np.array_equal(o["s_col"][:, :C].cpu().numpy(), s)
    if rowwise:
        qr, sr = Q.quantize_1x128_rowwise(bits)
        assert np.array_equal(o["q_row"].cpu().numpy(), qr)
        assert np.array_equal(o["s_row"][:, :R].cpu().numpy(), sr)


def test_quantize_grouped_columns_not_of_128(cuda_lib):
    fq = cuda_lib
    counts, C = [5, 0, 200], 176
    x = workloads.normal_bf16((sum(counts), C), 1.0, 52)
    o = fq.quantize_1x128_grouped(x.cuda(), offsets(counts))
    q, s = padded_oracle(workloads.bf16_bits(x), counts, fq.fp8q_grouped_capacity(sum(counts), 3))
    assert np.array_equal(o["q_col"].cpu().numpy(), q) and np.array_equal(o["s_col"][:, :C].cpu().numpy(), s)


@pytest.mark.parametrize("offs", [[0, 200, 100, 300], [0, 100, 100000, 300], [0, -5, 200, 300], [0, 10, 20, 250]])
def test_quantize_grouped_offsets_out_of_rule(cuda_lib, offs):
    fq = cuda_lib
    x = workloads.normal_bf16((300, 128), 1.0, 53).cuda()
    assert fq.device_status() == fq.FP8Q_OK
    fq.quantize_1x128_grouped(x, torch.tensor(offs, dtype=torch.int32, device="cuda"), rowwise=True)
    assert fq.device_status() == fq.FP8Q_ERR_DEVICE_ARG


def test_quantize_grouped_many_tiles_per_cta(cuda_lib):
    """Enough tiles that a CTA takes several columns of a band: against the ungrouped quantizer."""
    fq = cuda_lib
    counts, C = [1024, 128, 0, 4096, 256], 16384 + 128
    x = workloads.normal_bf16((sum(counts), C), 1.0, 54, device="cuda")
    o = fq.quantize_1x128_grouped(x, offsets(counts), rowwise=True)
    r = fq.quantize_1x128(x, rowwise=True, colwise=True)
    n = sum(counts)
    assert torch.equal(o["q_row"], r["q_row"]) and torch.equal(o["s_row"][:, :n], r["s_row"][:, :n])
    assert torch.equal(o["q_col"][:, :n], r["q_col"]) and torch.equal(o["s_col"][:n // 128, :C], r["s_col"][:, :C])
    assert bool((o["q_col"][:, n:] == 0).all()) and bool((o["s_col"][n // 128:, :C] == 1).all())


# ------------------------------------------------------------------------------ together
def test_expert_layer_step(cuda_lib):
    """Forward, both gradients and the accumulated main gradient of one expert projection, as a step
    uses them, from BF16 inputs: against 64-bit products of the dequantized operands."""
    fq = cuda_lib
    counts, Kin, Nout = [70, 0, 129, 300], 384, 256
    R, G = sum(counts), len(counts)
    X = workloads.normal_bf16((R, Kin), 1.0, 61, device="cuda")
    W = workloads.normal_bf16((G, Kin, Nout), 0.02, 62, device="cuda")
    dY = workloads.normal_bf16((R, Nout), 1e-3, 63, device="cuda")
    offs = offsets(counts)
    qw = fq.quantize_128x128_grouped(W)
    qx = fq.quantize_1x128_grouped(X, offs, rowwise=True)
    qy = fq.quantize_1x128_grouped(dY, offs, rowwise=True)
    main = torch.randn((G, Kin, Nout), device="cuda")
    before = main.double()
    y = fq.gemm(qx["q_row"], qw["q_t"], a_scale=qx["s_row"], b_scale=qw["s"], m_offsets=offs)
    dx = fq.gemm(qy["q_row"], qw["q"], layout=fq.FP8Q_DGRAD, a_scale=qy["s_row"], b_scale=qw["s"], m_offsets=offs)
    fq.gemm(qx["q_col"], qy["q_col"], layout=fq.FP8Q_WGRAD, a_scale=qx["s_col"], b_scale=qy["s_col"], m_offsets=offs,
            out=main, accumulate_fp32=True)
    assert fq.device_status() == fq.FP8Q_OK
    ref, t = rows_reference(qx["q_row"], qx["s_row"], qw["q_t"], qw["s"], counts, False)
    assert_within(y, ref, gamma(3) * t + 2.0 ** -8 * (ref.abs() + gamma(3) * t), "forward")
    ref, t = rows_reference(qy["q_row"], qy["s_row"], qw["q"], qw["s"], counts, True)
    assert_within(dx, ref, gamma(2) * t + 2.0 ** -8 * (ref.abs() + gamma(2) * t), "dgrad")
    ref, t = wgrad_reference(qx["q_col"], qx["s_col"], qy["q_col"], qy["s_col"], counts)
    assert_within(main, ref + before, gamma(3) * t + 2.0 ** -24 * (before.abs() + ref.abs() + gamma(3) * t), "wgrad")
    # and near the gradient in BF16 operands: every operand is within 2^-4 of itself
    at = 0
    for e, n in enumerate(counts):
        x, d = X[at:at + n].double(), dY[at:at + n].double()
        # codes are off by at most 2^-4 of the value or half a subnormal step (2^-10) of the tile's scale
        bound = 2.0 * (2.0 ** -4 + 2.0 ** -8) * (x.abs().t() @ d.abs()) + 2.0 ** -10 / 448 * n * (
            float(x.abs().max() if n else 0) * float(d.abs().max() if n else 0)) * 4 + 1e-6 * before[e].abs()
        assert float(((main[e].double() - before[e]) - x.t() @ d).abs().sub(bound).max()) <= 0
        at += n


def test_step_captured_and_replayed_with_other_routing(cuda_lib):
    """A captured step reads the offsets on the device: replayed with another routing it computes that one, next
    to the same step run eagerly on another stream."""
    fq = cuda_lib
    R, Kin, Nout, G = 600, 256, 384, 4
    W = workloads.normal_bf16((G, Kin, Nout), 0.02, 5, device="cuda")
    qw = fq.quantize_128x128_grouped(W)
    X, dY = torch.empty((R, Kin), dtype=torch.bfloat16, device="cuda"), torch.empty((R, Nout), dtype=torch.bfloat16,
                                                                                   device="cuda")
    offs = offsets([R, 0, 0, 0])
    main = torch.zeros((G, Kin, Nout), device="cuda")

    def step(X, dY, offs, main, stream=None):
        qx = fq.quantize_1x128_grouped(X, offs, rowwise=True, stream=stream)
        qy = fq.quantize_1x128_grouped(dY, offs, rowwise=True, stream=stream)
        y = fq.gemm(qx["q_row"], qw["q_t"], a_scale=qx["s_row"], b_scale=qw["s"], m_offsets=offs, stream=stream)
        dx = fq.gemm(qy["q_row"], qw["q"], layout=fq.FP8Q_DGRAD, a_scale=qy["s_row"], b_scale=qw["s"], m_offsets=offs,
                     stream=stream)
        fq.gemm(qx["q_col"], qy["q_col"], layout=fq.FP8Q_WGRAD, a_scale=qx["s_col"], b_scale=qy["s_col"],
                m_offsets=offs, out=main, accumulate_fp32=True, stream=stream)
        return y, dx

    def fill(seed, counts):
        X.copy_(workloads.normal_bf16((R, Kin), 1.0, seed, device="cuda"))
        dY.copy_(workloads.normal_bf16((R, Nout), 1e-3, seed + 1, device="cuda"))
        offs.copy_(offsets(counts))
        main.zero_()

    fill(1, [R, 0, 0, 0])
    step(X, dY, offs, main)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, dx = step(X, dY, offs, main)
    side = torch.cuda.Stream()
    for seed, counts in ((11, [1, 0, 599, 0]), (21, [150, 151, 149, 150]), (31, [0, 0, 0, 600])):
        fill(seed, counts)
        other = [t.clone() for t in (X, dY, offs)]
        main2 = torch.zeros_like(main)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            y2, dx2 = step(*other, main2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(main, main2)
        qx = fq.quantize_1x128_grouped(X, offs, rowwise=True)
        ref, t = rows_reference(qx["q_row"], qx["s_row"], qw["q_t"], qw["s"], counts, False)
        assert_within(y, ref, gamma(2) * t + 2.0 ** -8 * (ref.abs() + gamma(2) * t), "replayed")
    assert fq.device_status() == fq.FP8Q_OK


def test_two_host_threads(cuda_lib):
    """Two threads, each with its own stream and tensors, get the results of one."""
    import threading
    fq = cuda_lib
    jobs = []
    for k in range(2):
        counts = [[40, 90, 3], [200, 0, 700]][k]
        a, b = codes((sum(counts), 384), 100 + k), codes((3, 256, 384), 200 + k)
        sa, sb = scales((3, sum(counts) + -sum(counts) % 4), 300 + k), scales((3, 2, 3), 400 + k)
        x = workloads.normal_bf16((sum(counts), 256), 1.0, 500 + k, device="cuda")
        jobs.append((a, b, sa, sb, offsets(counts), x))

    def work(job, out):
        a, b, sa, sb, offs, x = job
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                c = fq.gemm(a, b, a_scale=sa, b_scale=sb, m_offsets=offs)
                q = fq.quantize_1x128_grouped(x, offs)
                n = fq.clip_grad_norm([x], 1.0, out=[torch.empty_like(x)])
            torch.cuda.current_stream().synchronize()
        out += [c, q["q_col"], q["s_col"], n]

    alone = [[] for _ in jobs]
    for j, o in zip(jobs, alone):
        work(j, o)
    both = [[] for _ in jobs]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(j, o)) for j, o in zip(jobs, both)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for p, q in zip(alone, both):
        assert len(q) == 4 and all(torch.equal(u, v) for u, v in zip(p, q))


def test_results_are_not_taken_from_memory_that_another_stream_still_uses(cuda_lib):
    """Memory freed on the current stream, whose last kernel there has not run yet, is not handed to a call on
    another stream: its late write would land in that call's result."""
    fq = cuda_lib
    a, b, sa, sb = codes((600, 256), 1), codes((2, 256, 256), 2), scales((2, 600), 3), scales((2, 2, 2), 4)
    x = workloads.normal_bf16((600, 256), 1.0, 5, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    offs = offsets([300, 300])
    side = torch.cuda.Stream()
    calls = {
        "gemm": lambda s: [fq.gemm(a, b, a_scale=sa, b_scale=sb, m_offsets=offs, stream=s)],
        "quantize": lambda s: list(fq.quantize_1x128_grouped(x, offs, rowwise=True, stream=s).values()),
        "norm": lambda s: list(fq.norm_residual(x, x, w, w, w, quantize=True, stream=s).values()),
        "clip": lambda s: [fq.clip_grad_norm([x], 1.0, out=[y], stream=s)],
    }
    y = torch.empty_like(x)
    r = fq.norm_residual(x, x, w, w, w)
    calls["backward"] = lambda s: list(fq.norm_residual_backward(x, x, x, r["h"], r["rstd_pre"], w, w, r["rstd_post"],
                                                                 w, stream=s).values())
    for name, call in calls.items():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        sizes = [t.untyped_storage().nbytes() for t in call(None)]
        torch.cuda.synchronize()
        old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda._sleep(200_000_000)                       # about a tenth of a second
        for t in old:
            t.fill_(0x7F)
        del old, t
        got = call(side)
        torch.cuda.synchronize()
        for u, v in zip(want, got):
            if name == "quantize" and u.dtype == torch.float32:
                u, v = u[:, :256], v[:, :256]
            assert torch.equal(u, v), name
