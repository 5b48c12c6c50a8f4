"""The norms around a block, its gate and residual scale, and their gradients, against 64 bits.

Tolerances, with u = 2^-24 (one FP32 rounding).  A row sum adds at most 32 terms per thread, 5
levels over a warp and 5 over up to 16 warps, so with one more rounding per term its error is below
54 u of the sum of magnitudes: rms(y), half of that and four roundings more, is within 32 u of
itself, and
  h' = alpha h + gate z   is within  E_h = u (2 |alpha h| + 40 |gate z|),
  rms(h')                 within     32 u + ||E_h|| / ||h'||  of itself (it moves with the norm of h'),
  n                       within     E_n = |w_pre| rms(h') E_h + (36 u + ||E_h|| / ||h'||) |n|.
Backward, the same counts: with m(v) the row mean of |v|,
  d    within  D = 70 u (|dh'| + rstd (|a| + |xh| m(a xh))),
  dy   within  rstd_post (|gate w_post| D + |yh| m(gate w_post yh D)) + 70 u rstd_post (|b| + |yh| m(b yh)),
  a column sum of R terms within (R + 24) u times the sum of magnitudes, plus what the terms carry.
Stored values add half a step of their type; E4M3 codes 2^-4 of the value or half a subnormal step
(2^-10) of the tile's scale."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
B, F = torch.bfloat16, torch.float32


def inputs(R, C, hd, wd, post, gate, seed=0, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def mat(sigma, dt):
        m = torch.full((R, C + pad), float("nan"), dtype=dt, device="cuda")[:, :C]
        return m.copy_(torch.randn((R, C), generator=g, device="cuda") * sigma)

    vec = lambda a, b: (a + b * torch.randn(C, generator=g, device="cuda")).to(wd)  # noqa: E731
    return dict(y=mat(0.7, B), h=mat(1.5, hd), w_pre=vec(1, 0.2), w_post=vec(1, 0.2) if post else None,
                gate=vec(0, 0.5) if gate else None, dn=mat(1e-2, B), dh=mat(1e-2, hd))


def forward64(x, alpha, eps):
    y, h = x["y"].double(), x["h"].double()
    rq = None
    z = y
    if x["w_post"] is not None:
        rq = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        z = y * rq * x["w_post"].double()
    if x["gate"] is not None:
        z = z * x["gate"].double()
    hp = alpha * h + z
    rp = 1 / torch.sqrt((hp * hp).mean(1, keepdim=True) + eps)
    n = hp * rp * x["w_pre"].double()
    eh = U * (2 * (alpha * h).abs() + 40 * z.abs())
    move = eh.norm(dim=1, keepdim=True) / hp.norm(dim=1, keepdim=True).clamp(min=1e-300)
    en = x["w_pre"].double().abs() * rp * eh + (36 * U + move) * n.abs()
    return dict(h=hp, n=n, rp=rp, rq=rq, eh=eh, en=en, er=(32 * U + move) * rp)


def within(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() - bound).max() if got.numel() else torch.zeros(())
    assert float(over) <= 0, f"{what}: {float(over)} over the bound"


def check_forward(x, o, alpha, eps, hd):
    r = forward64(x, alpha, eps)
    R, C = x["y"].shape
    within(o["h"], r["h"], r["eh"] + HALF[hd] * (r["h"].abs() + r["eh"]), "h")
    within(o["rstd_pre"], r["rp"].view(-1), r["er"].view(-1), "rstd_pre")
    if r["rq"] is not None:
        within(o["rstd_post"], r["rq"].view(-1), 32 * U * r["rq"].view(-1), "rstd_post")
    else:
        assert o["rstd_post"] is None
    if "n" in o:
        within(o["n"], r["n"], r["en"] + HALF[B] * (r["n"].abs() + r["en"]), "n")
    if "q_row" in o:
        tiles = r["n"].view(R, C // 128, 128)
        s = o["s_row"][:, :R].t().double()
        amax, err = tiles.abs().amax(2), r["en"].view(R, C // 128, 128).amax(2)
        empty = amax == 0
        within(torch.where(empty, s.new_zeros(()), s), amax / 448, err / 448 + 3 * U * (amax + err) / 448, "scales")
        assert bool((s[empty] == 1).all())
        v = o["q_row"].view(torch.float8_e4m3fn).double().view(R, C // 128, 128) * s[:, :, None]
        e = r["en"].view(R, C // 128, 128)
        # 448 s may fall short of the largest value by the roundings of s (3 u): saturation
        within(v, tiles, e + (2.0 ** -4 + 4 * U) * (tiles.abs() + e) + 2.0 ** -10 * s[:, :, None], "codes")
    return r


SHAPES = [(1, 8), (3, 256), (1, 16384), (5, 7168), (2, 16376), (700, 128), (333, 1000), (64, 4096), (150, 4104),
          (301, 8192), (149, 8200), (450, 9344), (450, 9352), (310, 14336), (460, 16384)]


@pytest.mark.parametrize("post,gate", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("hd,wd", [(B, B), (B, F), (F, B), (F, F)])
@pytest.mark.parametrize("R,C", SHAPES)
def test_forward(cuda_lib, R, C, hd, wd, post, gate):
    x = inputs(R, C, hd, wd, post, gate, seed=R + C)
    args = (x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"])
    o = cuda_lib.norm_residual(*args, alpha=0.9, eps=1e-5, normed=True, quantize=C % 128 == 0)
    check_forward(x, o, 0.9, 1e-5, hd)
    if C % 128 == 0:
        q = cuda_lib.norm_residual(*args, alpha=0.9, eps=1e-5, normed=False, quantize=True)
        assert "n" not in q and torch.equal(q["q_row"], o["q_row"]) and torch.equal(q["h"], o["h"])
    assert cuda_lib.device_status() == 0


def test_forward_strides_in_place_and_stream(cuda_lib):
    """Padded rows, h' over h, on a stream of its own."""
    x = inputs(77, 640, F, B, True, True, seed=5, pad=24)
    keep = x["h"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], alpha=0.5, out=x["h"], quantize=True,
                               stream=s)
    s.synchronize()
    assert o["h"] is x["h"]
    check_forward({**x, "h": keep}, o, 0.5, 1e-6, F)


def test_zero_rows_and_zero_values(cuda_lib):
    x = inputs(0, 256, B, B, True, True)
    o = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], quantize=True)
    assert o["h"].shape == (0, 256) and o["n"].shape == (0, 256)
    x = inputs(3, 256, B, B, True, False)
    x["y"].zero_()
    x["h"][1].zero_()
    o = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], None, eps=1e-6, quantize=True)
    check_forward(x, o, 1.0, 1e-6, B)
    assert bool((o["h"][1] == 0).all()) and bool((o["n"][1] == 0).all()) and bool((o["q_row"][1] == 0).all())


def test_nan_stays_in_its_row(cuda_lib):
    x = inputs(9, 512, F, F, True, True)
    clean = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"])
    x["h"][4, 7] = float("nan")
    x["y"][6, 3] = float("inf")
    o = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"])
    rest = [r for r in range(9) if r not in (4, 6)]
    assert torch.equal(o["n"][rest], clean["n"][rest]) and torch.equal(o["h"][rest], clean["h"][rest])
    assert bool(o["n"][4].isnan().all()) and bool(o["n"][6].isnan().any())


def backward64(x, r, alpha):
    """x with h the stored h', and rstd of r: the formula, and the bounds of the module's text."""
    C = x["y"].shape[1]
    R = x["y"].shape[0]
    one = torch.ones(C, dtype=torch.float64, device="cuda")
    w = x["w_pre"].double()
    rp = r["rstd_pre"].double()[:, None]
    xh, dn, dh = x["h"].double() * rp, x["dn"].double(), x["dh"].double()
    a = dn * w
    d = dh + rp * (a - xh * (a * xh).mean(1, keepdim=True))
    D = 70 * U * (dh.abs() + rp * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True)))
    y = x["y"].double()
    gate = one if x["gate"] is None else x["gate"].double()
    out = {"dh": (alpha * d, abs(alpha) * D + U * (alpha * d).abs())}
    col = lambda t, e: (t.sum(0), (R + 24) * U * t.abs().sum(0) + e.sum(0))  # noqa: E731
    out["dw_pre"] = col(dn * xh, 3 * U * (dn * xh).abs())
    if x["w_post"] is None:
        out["dy"] = (gate * d, gate.abs() * D + U * (gate * d).abs())
        wq, yh = one, y
    else:
        wq = x["w_post"].double()
        rq = r["rstd_post"].double()[:, None]
        yh = y * rq
        b = d * gate * wq
        gw = (gate * wq).abs()
        out["dy"] = (rq * (b - yh * (b * yh).mean(1, keepdim=True)),
                     rq * (gw * D + yh.abs() * (gw * yh.abs() * D).mean(1, keepdim=True))
                     + 70 * U * rq * (b.abs() + yh.abs() * (b * yh).abs().mean(1, keepdim=True)))
        s, e = col(d * yh, D * yh.abs() + 3 * U * (d * yh).abs())
        out["dw_post"] = (s * gate, (e + U * s.abs()) * gate.abs())
    if x["gate"] is not None:
        s, e = col(d * yh, D * yh.abs() + 3 * U * (d * yh).abs())
        out["dgate"] = (s * wq, (e + U * s.abs()) * wq.abs())
    return out


def check_backward(x, r, o, alpha):
    want = backward64(x, r, alpha)
    assert set(o) == set(want)
    for k, (v, e) in want.items():
        half = HALF[o[k].dtype]
        within(o[k], v, e + half * (v.abs() + e), k)


def run_backward(fq, x, r, alpha, **kw):
    return fq.norm_residual_backward(x["dn"], x["dh"], x["y"], x["h"], r["rstd_pre"], x["w_pre"], x["w_post"],
                                     r["rstd_post"], x["gate"], alpha=alpha, **kw)


@pytest.mark.parametrize("post,gate", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("hd,wd", [(B, B), (B, F), (F, B), (F, F)])
@pytest.mark.parametrize("R,C", SHAPES)
def test_backward(cuda_lib, R, C, hd, wd, post, gate):
    x = inputs(R, C, hd, wd, post, gate, seed=R + C)
    r = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], alpha=0.9, eps=1e-5)
    x["h"] = r["h"]
    o = run_backward(cuda_lib, x, r, 0.9)
    check_backward(x, r, o, 0.9)
    again = run_backward(cuda_lib, x, r, 0.9)
    assert all(torch.equal(o[k], again[k]) for k in o)
    assert cuda_lib.device_status() == 0


def test_backward_zero_rows(cuda_lib):
    x = inputs(0, 256, F, F, True, True)
    r = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"])
    x["h"] = r["h"]
    o = run_backward(cuda_lib, x, r, 1.0)
    assert all(bool((o[k] == 0).all()) for k in ("dw_pre", "dw_post", "dgate")) and o["dy"].shape == (0, 256)


def test_backward_strides_and_stream(cuda_lib):
    x = inputs(200, 1152, B, F, True, True, seed=8, pad=8)
    r = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"])
    x["h"] = r["h"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = run_backward(cuda_lib, x, r, 1.0, stream=s)
    s.synchronize()
    check_backward(x, r, o, 1.0)


@pytest.mark.parametrize("post,gate", [(True, True), (False, True), (True, False)])
def test_backward_against_differences(cuda_lib, post, gate):
    """Directional derivatives of sum(n cn) + sum(h' ch), by central differences of the 64-bit forward
    pass, against the kernel's gradients.  Step t: the difference is off by t^2 times a third
    derivative (about 1e-8 of the scale here) and 1e-16 / t; the gradients by the bounds above."""
    R, C, alpha, eps, t = 6, 256, 0.8, 1e-5, 1e-4
    x = inputs(R, C, F, F, post, gate, seed=3)
    r = cuda_lib.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], alpha=alpha, eps=eps)
    stored = {**x, "h": r["h"]}
    o = run_backward(cuda_lib, stored, r, alpha)
    bounds = backward64(stored, r, alpha)
    g = torch.Generator(device="cuda").manual_seed(9)
    names = {"y": "dy", "h": "dh", "w_pre": "dw_pre", "w_post": "dw_post", "gate": "dgate"}

    def loss(z):
        f = forward64(z, alpha, eps)
        return float((f["n"] * x["dn"].double()).sum() + (f["h"] * x["dh"].double()).sum())

    for name, grad in names.items():
        if x[name] is None:
            continue
        v = torch.randn(x[name].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = ({**x, name: x[name].double() + s * v} for s in (t, -t))
        diff = (loss(plus) - loss(minus)) / (2 * t)
        val, e = bounds[grad]
        half = HALF[o[grad].dtype]
        # the kernel's h' is rounded (FP32) where the formula's is not: 40 u of every term more
        slack = float(((e + (half + 400 * U) * val.abs()) * v.abs()).sum()) + 1e-6 * float((val * v).abs().sum())
        assert abs(diff - float((o[grad].double() * v).sum())) <= slack, name


@pytest.mark.parametrize("C", [256, 3200, 4096, 7168, 8200, 16384])
def test_a_row_does_not_depend_on_the_others(cuda_lib, C):
    """The same row among 3 and among 500 rows, to the bit, forward and backward."""
    fq = cuda_lib
    x = inputs(500, C, F, B, True, True, seed=7)
    r = fq.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], quantize=C % 128 == 0)
    few = {k: v[:3] if v is not None and v.dim() == 2 else v for k, v in x.items()}
    rf = fq.norm_residual(few["y"], few["h"], x["w_pre"], x["w_post"], x["gate"], quantize=C % 128 == 0)
    for k in ("h", "n", "rstd_pre", "rstd_post") + (("q_row",) if C % 128 == 0 else ()):
        assert torch.equal(r[k][:3], rf[k]), k
    o = run_backward(fq, {**x, "h": r["h"]}, r, 1.0)
    of = run_backward(fq, {**few, "h": rf["h"]}, rf, 1.0)
    assert torch.equal(o["dh"][:3], of["dh"]) and torch.equal(o["dy"][:3], of["dy"])


def test_more_than_2_31_values(cuda_lib):
    """Rows past 32-bit element offsets equal the same rows alone."""
    R, C = 270_000, 8192                                   # 2.2e9 values
    y = torch.randn((64, C), device="cuda").to(B).repeat(R // 64 + 1, 1)[:R]
    h = torch.randn((64, C), device="cuda").to(B).repeat(R // 64 + 1, 1)[:R]
    w = torch.ones(C, dtype=B, device="cuda")
    o = cuda_lib.norm_residual(y, h, w, w, None, normed=False, quantize=True)
    few = cuda_lib.norm_residual(y[-200:], h[-200:], w, w, None, normed=False, quantize=True)
    assert torch.equal(o["q_row"][-200:], few["q_row"]) and torch.equal(o["h"][-200:], few["h"])
    assert torch.equal(o["s_row"][:, R - 200:R], few["s_row"][:, :200])
    del o
    dn = y
    g = cuda_lib.norm_residual_backward(dn, h, y, h, torch.ones(R, device="cuda"), w, alpha=0.5)
    last = cuda_lib.norm_residual_backward(dn[-200:], h[-200:], y[-200:], h[-200:], torch.ones(200, device="cuda"), w,
                                           alpha=0.5)
    assert torch.equal(g["dh"][-200:], last["dh"]) and torch.equal(g["dy"][-200:], last["dy"])


def test_graph_beside_an_eager_call(cuda_lib):
    """Forward and backward captured together and replayed on new values, with an eager backward of
    other values in between; the graphs' workspaces are their own."""
    fq = cuda_lib
    x, z = inputs(130, 512, F, F, True, True, seed=1), inputs(130, 512, F, F, True, True, seed=2)

    def step(x):
        r = fq.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], alpha=0.9, quantize=True)
        return r, run_backward(fq, {**x, "h": r["h"]}, r, 0.9)

    step(x)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(x)
        graphs.append((g, out))
    for seed in (11, 12):
        new = inputs(130, 512, F, F, True, True, seed=seed)
        for k in x:
            x[k].copy_(new[k])
        for g, _ in graphs:
            g.replay()
        rz, oz = step(z)
        torch.cuda.synchronize()
        for _, (r, o) in graphs:
            check_forward(x, r, 0.9, 1e-6, F)
            check_backward({**x, "h": r["h"]}, r, o, 0.9)
        check_backward({**z, "h": rz["h"]}, rz, oz, 0.9)


def test_norm_into_the_quantized_product(cuda_lib):
    """norm -> FP8 product, the way a block uses it: codes and scales feed gemm() as they are."""
    fq = cuda_lib
    x = inputs(200, 512, B, B, True, True, seed=4)
    o = fq.norm_residual(x["y"], x["h"], x["w_pre"], x["w_post"], x["gate"], normed=False, quantize=True)
    w = torch.randn((512, 256), device="cuda").mul_(0.02).to(B)
    qw = fq.quantize_128x128(w)
    c = fq.gemm(o["q_row"], qw["q_t"], a_scale=o["s_row"], b_scale=qw["s"])
    a = o["q_row"].view(torch.float8_e4m3fn).double() * o["s_row"][:, :200].double().t().repeat_interleave(128, 1)
    b = qw["q_t"].view(torch.float8_e4m3fn).double() * qw["s"].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    gamma = 128 * 2.0 ** -23 + 7 * U
    ref, t = a @ b.t(), a.abs() @ b.abs().t()
    within(c, ref, gamma * t + 2.0 ** -8 * (ref.abs() + gamma * t), "product")
