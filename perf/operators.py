"""The operators around an expert (MoE) training or serving step, as one pass each:

  rows      products grouped by expert over ragged rows: C[r] = A[r] . B_e^T for the rows r of expert e
            (forward of few rows, as in decoding, and the gradient of the activations)
  wgrad     products grouped by expert over ragged tokens: C_e (+)= X_e^T . dY_e
  quantize  1x128 quantization whose transposed output keeps every expert's tokens in tiles of their own
  clip      global norm of many gradient tensors, and their clipped copies
  norm_fwd  h' = alpha h + gate * norm(y), then the next block's norm of h', quantized or in BF16
  norm_bwd  its gradients

Operands of the products are E4M3 codes with FP32 decode scales: 1x128 tiles for activations and
gradients, 128x128 blocks for weights.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
EPS_CLIP, EPS_NORM = 1e-6, 1e-5


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one request through the up projection of its 8 experts
        dict(name="rows decode 1 token", op="rows", layout="fprop", tokens=1, topk=8, experts=32, K=7168, N=2048,
             skew=0.4),
        # a decoding batch: a few rows for nearly every expert
        dict(name="rows decode 24 tokens", op="rows", layout="fprop", tokens=24, topk=8, experts=32, K=2048, N=7168,
             skew=0.4),
        # activation gradient of the down projection, one micro-batch, experts loaded unevenly
        dict(name="rows dgrad 2048 tokens", op="rows", layout="dgrad", tokens=2048, topk=8, experts=32, K=7168,
             N=2048, skew=1.1),
        # activation gradient of the up projection, a long micro-batch
        dict(name="rows dgrad 8192 tokens", op="rows", layout="dgrad", tokens=8192, topk=8, experts=32, K=2048,
             N=7168, skew=0.4),
        # weight gradient of a small odd-sized layer into a BF16 gradient, most experts with a partial tile
        dict(name="wgrad odd 1000 tokens", op="wgrad", tokens=1000, topk=2, experts=8, M=1040, N=528, skew=1.1,
             accumulate=False),
        # weight gradient of the down projection accumulated into FP32 main gradients
        dict(name="wgrad 4096 tokens", op="wgrad", tokens=4096, topk=8, experts=32, M=2048, N=7168, skew=0.4,
             accumulate=True),
        # routed activations of a micro-batch: forward operand and weight-gradient operand in one read
        dict(name="quantize 4096 tokens", op="quantize", tokens=4096, topk=4, experts=32, cols=7168, skew=0.4),
        # gradients of a small module: 12 tensors, odd sizes
        dict(name="clip 12 tensors", op="clip", tensors=12, f32=90001, bf16=10003, scaled=True),
        # main gradients of a few layers and BF16 gradients of the rest
        dict(name="clip 300 tensors", op="clip", tensors=300, f32=400000003, bf16=100000001, scaled=True),
        # one decoding step of a few sequences, into the next FP8 product
        dict(name="norm_fwd 4 rows", op="norm_fwd", rows=4, cols=7168, post=True, gate=True, quant=True, h32=False,
             w32=False),
        # a training micro-batch, FP32 residual stream, into the next FP8 product
        dict(name="norm_fwd 8192 rows", op="norm_fwd", rows=8192, cols=7168, post=True, gate=True, quant=True,
             h32=True, w32=True),
        # its gradients
        dict(name="norm_bwd 8192 rows", op="norm_bwd", rows=8192, cols=7168, post=True, gate=True, h32=True, w32=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rows", "rows", "wgrad", "quantize", "clip", "norm_fwd", "norm_bwd"))
    if op in ("rows", "wgrad", "quantize"):
        experts = rng.choice((1, 3, 8, 17, 32, 64))
        c = dict(op=op, tokens=_log(rng, 1, 8192), topk=rng.randint(1, min(8, experts)), experts=experts,
                 skew=round(rng.uniform(0.0, 1.1), 3))
        if op == "rows":
            c.update(layout=rng.choice(("fprop", "dgrad")), K=128 * _log(rng, 2, 56), N=128 * _log(rng, 1, 56))
            while c["experts"] * c["K"] * c["N"] > 32 * 2048 * 7168:
                c["K"] = 128 * max(1, c["K"] // 256)
        elif op == "wgrad":
            c.update(M=16 * _log(rng, 8, 448), N=16 * _log(rng, 8, 448), accumulate=rng.random() < 0.5)
            while c["experts"] * c["M"] * c["N"] > 32 * 2048 * 7168:
                c["M"] = 16 * max(8, c["M"] // 32)
            c["tokens"] = min(c["tokens"], 4096)
        else:
            c.update(cols=128 * _log(rng, 1, 56))
            c["tokens"] = min(c["tokens"], 16384 // c["topk"])
        return c
    if op == "clip":
        f32, bf16 = _log(rng, 1, 4 * 10 ** 8), _log(rng, 1, 10 ** 8)
        return dict(op=op, tensors=2 + _log(rng, 1, 300), f32=f32, bf16=bf16, scaled=rng.random() < 0.7)
    c = dict(op=op, rows=_log(rng, 1, 8192), cols=128 * _log(rng, 2, 56), post=rng.random() < 0.7,
             gate=rng.random() < 0.7, h32=rng.random() < 0.5, w32=rng.random() < 0.5)
    if op == "norm_fwd":
        c["quant"] = rng.random() < 0.6
    if not c.get("quant") and rng.random() < 0.4:
        c["cols"] -= 8 * rng.randint(1, 15)
    return c


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).mul_(sigma).to(dtype)


def _route(case, g):
    """Row offsets of the experts (int32 on the device, and on the host): every token goes to `topk` distinct
    experts drawn with popularity (e + 1)^-skew."""
    E, k = case["experts"], case["topk"]
    p = (torch.arange(E, dtype=torch.float64, device=DEV) + 1.0) ** -case["skew"]
    choice = torch.multinomial(p.float().expand(case["tokens"], E).contiguous(), k, generator=g)
    counts = torch.bincount(choice.reshape(-1), minlength=E)
    offs = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offs[1:] = torch.cumsum(counts, 0)
    return offs.to(torch.int32), [int(v) for v in offs.cpu()]


def _tile_codes(x, dim):
    """E4M3 values and FP32 decode scales of the 128-long tiles of x (..., 128, ...) along `dim`."""
    amax = x.abs().amax(dim, keepdim=True)
    sf = torch.where(amax == 0, torch.ones_like(amax), 448.0 / amax).clamp(max=torch.finfo(torch.float32).max)
    return (x * sf).clamp(-448.0, 448.0).to(E4M3), (1.0 / sf).squeeze(dim)


def _block_codes(w):
    """128x128 blocks of w (G, N, K): codes (G, N, K) and decode scales (G, N/128, K/128)."""
    G, N, K = w.shape
    amax = w.abs().view(G, N // 128, 128, K // 128, 128).amax((2, 4), keepdim=True)
    sf = torch.where(amax == 0, torch.ones_like(amax), 448.0 / amax)
    q = (w.view(G, N // 128, 128, K // 128, 128) * sf).to(E4M3).view(G, N, K)
    return q.view(torch.uint8), (1.0 / sf).view(G, N // 128, K // 128)


def _capacity(rows, experts):
    """Tokens of the padded layout: every expert's tokens rounded up to a multiple of 128, at most."""
    return 128 * min(rows // 128 + experts, rows)


def _padded(offs, capacity):
    """For every place of the padded layout: its source row, and whether it holds one; and its expert."""
    offs = offs.to(torch.int64)
    ends = torch.cumsum((offs[1:] - offs[:-1] + 127) // 128 * 128, 0)
    p = torch.arange(capacity, device=DEV)
    e = torch.searchsorted(ends, p, right=True).clamp_(max=offs.numel() - 2)
    start = torch.cat((ends.new_zeros(1), ends[:-1]))
    row = offs[e] + p - start[e]
    return row, (row < offs[e + 1]) & (p < ends[-1]), e


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("rows", "wgrad", "quantize"):
        s["offs"], host = _route(case, g)
        rows = host[-1]
        # the longest expert's rows: what a program that pads its experts to one length knows
        s["longest"] = max(b - a for a, b in zip(host, host[1:]))
    if op == "rows":
        K, N, E = case["K"], case["N"], case["experts"]
        x = _normal(g, (rows, K), 1.0, torch.bfloat16).float()
        x[torch.rand(x.shape, generator=g, device=DEV) < 1e-3] *= 50.0
        q, sc = _tile_codes(x.view(rows, K // 128, 128), 2)
        s["a"] = q.view(torch.uint8).view(rows, K)
        s["a_scale"] = torch.ones((K // 128, rows + -rows % 4), device=DEV)
        s["a_scale"][:, :rows] = sc.t()
        w = _normal(g, (E, N, K), 0.02)
        s["b"], bs = _block_codes(w)
        s["b_scale"] = bs if case["layout"] == "fprop" else bs.transpose(1, 2).contiguous()
    elif op == "wgrad":
        cap = _capacity(rows, case["experts"])
        row, full, _ = _padded(s["offs"], cap)
        for name, width, sigma in (("x", case["M"], 1.0), ("dy", case["N"], 1e-3)):
            v = _normal(g, (rows, width), sigma, torch.bfloat16).float()
            v = torch.where(full[:, None], v[row.clamp(max=rows - 1)], v.new_zeros(()))
            q, sc = _tile_codes(v.view(cap // 128, 128, width), 1)
            s[name] = q.view(torch.uint8).view(cap, width).t().contiguous()
            s[name + "_scale"] = sc.contiguous()
        s["out"] = _normal(g, (case["experts"], case["M"], case["N"]), 1e-2) if case["accumulate"] else None
    elif op == "quantize":
        x = _normal(g, (rows, case["cols"]), 1.0)
        x[torch.rand(x.shape, generator=g, device=DEV) < 1e-3] *= 50.0
        s["x"] = x.to(torch.bfloat16)
    elif op == "clip":
        total = case["f32"] + case["bf16"]
        size = 1.0 / math.sqrt(total)                 # the gradients' norm is about 4 or about 1/4
        size *= 4.0 if case["scaled"] else 0.25
        s["max_norm"] = 1.0
        s["f32"] = _normal(g, (case["f32"],), size)
        s["bf16"] = _normal(g, (case["bf16"],), size, torch.bfloat16)
        s["f32_out"], s["bf16_out"] = torch.empty_like(s["f32"]), torch.empty_like(s["bf16"])
        # the tensors are pieces of two flat buffers, as main gradients are; their sizes spread widely
        r = random.Random(seed)
        s["grads"], s["outs"] = [], []
        for name, n in (("f32", max(1, case["tensors"] * 2 // 3)), ("bf16", max(1, case["tensors"] // 3))):
            w = [math.exp(r.uniform(0.0, 6.0)) for _ in range(n)]
            cuts, at = [0], 0.0
            for v in w:
                at += v
                cuts.append(min(case[name], int(case[name] * at / sum(w))))
            cuts[-1] = case[name]
            s["grads"] += [s[name][a:b] for a, b in zip(cuts, cuts[1:])]
            s["outs"] += [s[name + "_out"][a:b] for a, b in zip(cuts, cuts[1:])]
    else:
        R, C = case["rows"], case["cols"]
        hd, wd = (torch.float32 if case["h32"] else torch.bfloat16), (torch.float32 if case["w32"] else torch.bfloat16)
        s["alpha"] = 0.875
        s["y"] = _normal(g, (R, C), 0.6, torch.bfloat16)
        s["h"] = _normal(g, (R, C), 1.5, hd)
        s["w_pre"] = (1.0 + _normal(g, (C,), 0.1)).to(wd)
        s["w_post"] = (1.0 + _normal(g, (C,), 0.1)).to(wd) if case["post"] else None
        s["gate"] = _normal(g, (C,), 0.5, wd) if case["gate"] else None
        if op == "norm_bwd":
            h, _, _, rp, rq = _norm_plain(s)
            s["h"], s["rstd_pre"], s["rstd_post"] = h.to(hd), rp, rq
            s["dn"] = _normal(g, (R, C), 1e-3, torch.bfloat16)
            s["dh"] = _normal(g, (R, C), 1e-3, hd)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _values(codes):
    return codes.view(E4M3).float()


def _rows_plain(s):
    a, b, offs = s["a"], s["b"], s["offs"].to(torch.int64)
    rows, K = a.shape
    E, N, _ = b.shape
    x = (_values(a).view(rows, K // 128, 128) * s["a_scale"][:, :rows].t()[:, :, None]).view(rows, K)
    bs = s["b_scale"] if s["case"]["layout"] == "fprop" else s["b_scale"].transpose(1, 2)
    w = (_values(b).view(E, N // 128, 128, K // 128, 128) * bs[:, :, None, :, None]).view(E, N, K)
    place = torch.arange(s["longest"], device=DEV)
    at = (offs[:-1, None] + place).clamp(max=rows - 1)
    c = torch.bmm(x[at], w.transpose(1, 2))           # every expert's rows, padded to the longest
    r = torch.arange(rows, device=DEV)
    e = torch.searchsorted(offs[1:], r, right=True)
    return c[e, r - offs[e]].to(torch.bfloat16)


def _wgrad_plain(s):
    offs = s["offs"].to(torch.int64)
    E = offs.numel() - 1
    pad = (offs[1:] - offs[:-1] + 127) // 128 * 128
    ends = torch.cumsum(pad, 0)
    longest = (s["longest"] + 127) // 128 * 128
    place = torch.arange(longest, device=DEV)
    at = ((ends - pad)[:, None] + place).clamp(max=s["x"].shape[1] - 1)
    full = place < pad[:, None]

    def operand(q, sc):
        width, cap = q.shape
        v = (_values(q).view(width, cap // 128, 128) * sc.t()[:, :, None]).view(width, cap)
        v = v[:, at.view(-1)].view(width, E, longest) * full
        return v.transpose(0, 1)

    c = torch.bmm(operand(s["x"], s["x_scale"]), operand(s["dy"], s["dy_scale"]).transpose(1, 2))
    return s["out"].add_(c) if s["out"] is not None else c.to(torch.bfloat16)


def _quantize_plain(s):
    x = s["x"].float()
    rows, cols = x.shape
    q, sc = _tile_codes(x.view(rows, cols // 128, 128), 2)
    cap = _capacity(rows, s["case"]["experts"])
    row, full, _ = _padded(s["offs"], cap)
    v = torch.where(full[:, None], x[row.clamp(max=rows - 1)], x.new_zeros(()))
    qc, scc = _tile_codes(v.view(cap // 128, 128, cols), 1)
    return {"q_row": q.view(rows, cols), "s_row": sc.t().contiguous(), "q_col": qc.view(cap, cols).t().contiguous(),
            "s_col": scc}


def _clip_plain(s):
    norm = (s["f32"].double().square().sum() + s["bf16"].double().square().sum()).sqrt()
    coef = (s["max_norm"] / (norm + EPS_CLIP)).clamp(max=1.0).float()
    torch.mul(s["f32"], coef, out=s["f32_out"])
    s["bf16_out"].copy_(s["bf16"].float() * coef)
    return {"norm": norm.float(), "f32": s["f32_out"], "bf16": s["bf16_out"]}


def _norm_plain(s, t=torch.float32):
    """h' (unrounded), its norm (unrounded), the gated block output's norm factor and both rstd."""
    h, z = s["h"].to(t) * s["alpha"], s["y"].to(t)
    rq = None
    if s["w_post"] is not None:
        rq = (z.square().mean(1, keepdim=True) + EPS_NORM).rsqrt()
        z = z * rq * s["w_post"].to(t)
    h = h + (z if s["gate"] is None else z * s["gate"].to(t))
    rp = (h.square().mean(1, keepdim=True) + EPS_NORM).rsqrt()
    return h, h * rp * s["w_pre"].to(t), z, rp.view(-1), None if rq is None else rq.view(-1)


def _norm_fwd_plain(s):
    h, n, _, rp, rq = _norm_plain(s)
    out = {"h": h.to(s["h"].dtype), "rstd_pre": rp, "rstd_post": rq}
    if s["case"]["quant"]:
        R, C = n.shape
        q, sc = _tile_codes(n.view(R, C // 128, 128), 2)
        out.update(q_row=q.view(R, C), s_row=sc.t().contiguous())
    else:
        out["n"] = n.to(torch.bfloat16)
    return out


def _norm_bwd(s, t):
    """The gradients in arithmetic of type t, unrounded; sums over rows in 64 bits."""
    C = s["y"].shape[1]
    wp = s["w_pre"].to(t)
    rp = s["rstd_pre"].to(t)[:, None]
    xh, dn = s["h"].to(t) * rp, s["dn"].to(t)
    a = dn * wp
    d = s["dh"].to(t) + rp * (a - xh * ((a * xh).sum(1, keepdim=True) / C))
    out = {"dh": d * s["alpha"], "dw_pre": (dn * xh).sum(0, dtype=torch.float64)}
    gate = None if s["gate"] is None else s["gate"].to(t)
    dz = d if gate is None else d * gate
    y = s["y"].to(t)
    if s["w_post"] is None:
        out["dy"] = dz
        if gate is not None:
            out["dgate"] = (d * y).sum(0, dtype=torch.float64)
        return out
    w = s["w_post"].to(t)
    rq = s["rstd_post"].to(t)[:, None]
    yh = y * rq
    if gate is not None:
        out["dgate"] = (d * yh * w).sum(0, dtype=torch.float64)
    out["dw_post"] = (dz * yh).sum(0, dtype=torch.float64)
    b = dz * w
    out["dy"] = rq * (b - yh * ((b * yh).sum(1, keepdim=True) / C))
    return out


def _norm_bwd_plain(s):
    out = _norm_bwd(s, torch.float32)
    kinds = {"dh": s["h"].dtype, "dy": torch.bfloat16}
    return {k: v.to(kinds.get(k, torch.float32)) for k, v in out.items()}


# ------------------------------------------------------------------------------------ one pass
def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        return {"rows": _rows_plain, "wgrad": _wgrad_plain, "quantize": _quantize_plain, "clip": _clip_plain,
                "norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain}[op](state)
    import fp4_precision_gemm_b200 as fq
    if op == "rows":
        return fq.gemm(state["a"], state["b"], fq.FP8Q_BLOCKWISE,
                       fq.FP8Q_FPROP if case["layout"] == "fprop" else fq.FP8Q_DGRAD, a_scale=state["a_scale"],
                       b_scale=state["b_scale"], m_offsets=state["offs"])
    if op == "wgrad":
        return fq.gemm(state["x"], state["dy"], fq.FP8Q_BLOCKWISE, fq.FP8Q_WGRAD, a_scale=state["x_scale"],
                       b_scale=state["dy_scale"], m_offsets=state["offs"], out=state["out"],
                       accumulate_fp32=case["accumulate"])
    if op == "quantize":
        rows, cols = state["x"].shape
        o = fq.quantize_1x128_grouped(state["x"], state["offs"], rowwise=True, colwise=True)
        return {"q_row": o["q_row"].view(E4M3), "s_row": o["s_row"][:, :rows], "q_col": o["q_col"].view(E4M3),
                "s_col": o["s_col"][:, :cols]}
    if op == "clip":
        norm = fq.clip_grad_norm(state["grads"], state["max_norm"], eps=EPS_CLIP, out=state["outs"])
        return {"norm": norm, "f32": state["f32_out"], "bf16": state["bf16_out"]}
    if op == "norm_fwd":
        o = fq.norm_residual(state["y"], state["h"], state["w_pre"], w_post=state["w_post"], gate=state["gate"],
                             alpha=state["alpha"], eps=EPS_NORM, normed=not case["quant"], quantize=case["quant"])
        if case["quant"]:
            o["q_row"], o["s_row"] = o["q_row"].view(E4M3), o["s_row"][:, :case["rows"]]
        return o
    return fq.norm_residual_backward(state["dn"], state["dh"], state["y"], state["h"], state["rstd_pre"],
                                     state["w_pre"], w_post=state["w_post"], rstd_post=state["rstd_post"],
                                     gate=state["gate"], alpha=state["alpha"])


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once, weights of the experts that have
    rows (for few tokens: as many as even routing would hit)."""
    op = case["op"]
    if op in ("rows", "wgrad", "quantize"):
        rows, E = case["tokens"] * case["topk"], case["experts"]
        hit = E * (1.0 - (1.0 - case["topk"] / E) ** case["tokens"])
    if op == "rows":
        K, N = case["K"], case["N"]
        return {"bytes": rows * K * (1 + 1 / 32) + hit * N * K + 2 * rows * N, "flops": 2.0 * rows * N * K}
    if op == "wgrad":
        M, N = case["M"], case["N"]
        return {"bytes": rows * (M + N) * (1 + 1 / 32) + E * M * N * (8 if case["accumulate"] else 2),
                "flops": 2.0 * rows * M * N}
    if op == "quantize":
        C = case["cols"]
        return {"bytes": rows * C * (2 + 2 + 2 / 32), "flops": 4.0 * rows * C}
    if op == "clip":
        n = 4 * case["f32"] + 2 * case["bf16"]
        return {"bytes": 2.0 * n, "flops": 3.0 * (case["f32"] + case["bf16"])}
    n, h = case["rows"] * case["cols"], 4 if case["h32"] else 2
    if op == "norm_fwd":
        return {"bytes": n * (2 + 2 * h + (1 + 1 / 32 if case["quant"] else 2)), "flops": 12.0 * n}
    return {"bytes": n * (2 + 2 + 2 + 3 * h), "flops": 24.0 * n}


# ------------------------------------------------------------------------------------ 64 bits
def _e4m3_nearest(v):
    """Nearest E4M3 value (ties to even, saturating) of 64-bit v, from the format: 3 fraction bits, exponents from
    -6, subnormals below, largest 448."""
    m, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_tiles(x, dim):
    amax = x.abs().amax(dim, keepdim=True)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    return _e4m3_nearest(x / scale), scale.squeeze(dim)


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "rows":
        offs = [int(v) for v in s["offs"].cpu()]
        rows, N = s["a"].shape[0], case["N"]
        sa = s["a_scale"][:, :rows].to(f64).t().repeat_interleave(128, 1)
        bs = s["b_scale"] if case["layout"] == "fprop" else s["b_scale"].transpose(1, 2)
        c = torch.zeros((rows, N), dtype=f64, device=DEV)
        for e, (lo, hi) in enumerate(zip(offs, offs[1:])):
            w = s["b"][e].view(E4M3).to(f64) * bs[e].to(f64).repeat_interleave(128, 0).repeat_interleave(128, 1)
            c[lo:hi] = (s["a"][lo:hi].view(E4M3).to(f64) * sa[lo:hi]) @ w.t()
        return c
    if op == "wgrad":
        offs = [int(v) for v in s["offs"].cpu()]
        c = torch.zeros((case["experts"], case["M"], case["N"]), dtype=f64, device=DEV)
        at = 0
        for e, (lo, hi) in enumerate(zip(offs, offs[1:])):
            n = hi - lo
            end = at + (n + 127) // 128 * 128
            x, y = (s[k][:, at:at + n].contiguous().view(E4M3).to(f64)
                    * s[k + "_scale"].to(f64)[at // 128:end // 128].t().repeat_interleave(128, 1)[:, :n]
                    for k in ("x", "dy"))
            c[e] = x @ y.t()
            at = end
        return c if s["out"] is None else c + s["out"].to(f64)
    if op == "quantize":
        x = s["x"].to(f64)
        rows, cols = x.shape
        q, sc = _exact_tiles(x.view(rows, cols // 128, 128), 2)
        cap, offs = _capacity(rows, case["experts"]), [int(v) for v in s["offs"].cpu()]
        qc = torch.zeros((cols, cap), dtype=f64, device=DEV)
        scc = torch.ones((cap // 128, cols), dtype=f64, device=DEV)
        at = 0
        for lo, hi in zip(offs, offs[1:]):
            tiles = (hi - lo + 127) // 128
            v = torch.zeros((tiles * 128, cols), dtype=f64, device=DEV)
            v[:hi - lo] = x[lo:hi]
            if tiles:
                a, b = _exact_tiles(v.view(tiles, 128, cols), 1)
                qc[:, at * 128:(at + tiles) * 128] = a.view(tiles * 128, cols).t()
                scc[at:at + tiles] = b
            at += tiles
        return {"q_row": q.view(rows, cols), "s_row": sc.t().contiguous(), "q_col": qc, "s_col": scc}
    if op == "clip":
        norm = torch.sqrt(sum((s[k].to(f64) ** 2).sum() for k in ("f32", "bf16")))
        coef = min(1.0, s["max_norm"] / (float(norm) + EPS_CLIP))
        return {"norm": norm, "f32": s["f32"].to(f64) * coef, "bf16": s["bf16"].to(f64) * coef}
    C = case["cols"]
    rms = lambda v: 1.0 / torch.sqrt((v * v).sum(1) / C + EPS_NORM)  # noqa: E731
    y, w_pre = s["y"].to(f64), s["w_pre"].to(f64)
    one = torch.ones(C, dtype=f64, device=DEV)
    gate = one if s["gate"] is None else s["gate"].to(f64)
    w_post = one if s["w_post"] is None else s["w_post"].to(f64)
    if op == "norm_fwd":
        rq = rms(y) if case["post"] else None
        z = y * w_post * (1.0 if rq is None else rq[:, None])
        h = s["alpha"] * s["h"].to(f64) + gate * z
        rp = rms(h)
        n = h * rp[:, None] * w_pre
        out = {"h": h, "rstd_pre": rp, "rstd_post": rq}
        if case["quant"]:
            q, sc = _exact_tiles(n.view(-1, C // 128, 128), 2)
            out.update(q_row=q.view(-1, C), s_row=sc.t().contiguous())
        else:
            out["n"] = n
        return out
    # n_c = h_c rp w_c with rp a function of the whole row, and the same for y: the product rule, term by term
    rp = s["rstd_pre"].to(f64)[:, None]
    h, dn = s["h"].to(f64), s["dn"].to(f64)
    d = s["dh"].to(f64) + rp * w_pre * dn - h * rp ** 3 / C * (dn * w_pre * h).sum(1, keepdim=True)
    out = {"dh": s["alpha"] * d, "dw_pre": (dn * h * rp).sum(0)}
    if not case["post"]:
        out["dy"] = gate * d
        if case["gate"]:
            out["dgate"] = (d * y).sum(0)
        return out
    rq = s["rstd_post"].to(f64)[:, None]
    out["dy"] = rq * w_post * gate * d - y * rq ** 3 / C * (gate * d * w_post * y).sum(1, keepdim=True)
    out["dw_post"] = (gate * d * y * rq).sum(0)
    if case["gate"]:
        out["dgate"] = (d * w_post * y * rq).sum(0)
    return out
