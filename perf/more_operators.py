"""Measured cases of what stands around and between the expert products: the residual norm in front of an
expert layer (forward, into bf16 and 8 bits, and backward), tokens sorted by expert and back (with weights
and gradients), and the microscaled 4-bit (MXFP4) products with their quantizer and SwiGLU.

Each case has a plain form (elementary torch operations in fp32, rounded once at the end) and the library's
own calls; ``own`` chooses between them. Layer sizes are those of the layer families in ``synth.SHAPES``
(qwen36, dsv4, odd_h).

Slot s = t * k + j is token t's j-th expert. Rows sorted by expert: row p holds slot[p], expert e owns the
rows [offs[e], offs[e + 1]), and pos[t, j] is the row of slot t * k + j.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest scale of a block of 128
EPS = 1e-6
BLOCK = 64          # rows per batch entry of the plain products


def listed():
    return [
        # one token before an expert layer: bf16 for the router, 8 bits for the experts; latency
        dict(name="norm 1 token", op="norm", form="forward", rows=1, hidden=2048, residual="bf16", out="both", offset=1.0),
        # a training step's forward norm, with what its backward needs
        dict(name="norm 8192 tokens", op="norm", form="forward", rows=8192, hidden=2048, residual="bf16", out="bf16",
             offset=0.0),
        # prefill of a wide layer with an fp32 residual stream, an odd number of tokens, 8 bits only
        dict(name="norm wide 1999 tokens", op="norm", form="forward", rows=1999, hidden=4096, residual="f32", out="fp8",
             offset=0.0),
        # its gradient: through the norm and past it, and of the weight
        dict(name="norm backward 8192 tokens", op="norm", form="backward", rows=8192, hidden=2048, residual="bf16",
             past=True, offset=0.0),
        # an ordinary decode batch in 8 bits: 512 rows of codes and block scales
        dict(name="dispatch fp8 64 tokens", op="order", form="dispatch", tokens=64, top_k=8, experts=256, hidden=2048,
             type="fp8", skew=0.0),
        # a training step's gather, with the way back and the rows' weights
        dict(name="dispatch 8192 tokens", op="order", form="dispatch", tokens=8192, top_k=8, experts=256, hidden=2048,
             type="bf16", skew=1.1),
        # the end of a single-token step: eight rows into one, weighted; latency
        dict(name="combine 1 token", op="order", form="combine", tokens=1, top_k=8, experts=256, hidden=2048, type="f32",
             skew=0.0, add=True),
        # a training step's gradient of the weighted sum, of rows and weights
        dict(name="combine backward 8192 tokens", op="order", form="combine backward", tokens=8192, top_k=8, experts=256,
             hidden=2048, type="bf16", skew=1.1),
        # one token over 4-bit experts: SwiGLU into 4 bits and the down product, eight rows; latency
        dict(name="mxfp4 down 1 token", op="mxfp4", form="down", tokens=1, top_k=8, experts=256, n=2048, k=512, skew=0.0,
             out="bf16"),
        # decode batch over 4-bit experts
        dict(name="mxfp4 gate_up 64 tokens", op="mxfp4", form="product", tokens=64, top_k=8, experts=256, n=1024, k=2048,
             skew=0.0, out="bf16"),
        # prefill over 4-bit experts, skewed routing
        dict(name="mxfp4 gate_up 8192 tokens", op="mxfp4", form="product", tokens=8192, top_k=8, experts=256, n=1024,
             k=2048, skew=1.1, out="bf16"),
        # the plain 4-bit product: the wide layer's shared expert over a prefill chunk
        dict(name="mxfp4 shared 4096 tokens", op="mxfp4", form="product", tokens=4096, top_k=1, experts=1, n=4096, k=4096,
             skew=0.0, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "order", "order", "mxfp4", "mxfp4"])
    if op == "norm":
        form, residual = rng.choice(["forward", "forward", "backward"]), rng.choice(["none", "bf16", "f32"])
        case = dict(op="norm", form=form, rows=_log(rng, 1, 8192), residual=residual, offset=rng.choice([0.0, 1.0]))
        if form == "backward":
            return dict(case, hidden=_log(rng, 16, 4096), past=rng.random() < 0.5)
        out = rng.choice(["bf16", "fp8", "both"])
        return dict(case, out=out, hidden=_log(rng, 16, 4096) if out == "bf16" else 16 * _log(rng, 1, 256))
    experts = rng.choice([8, 60, 128, 256])
    top_k, tokens = rng.choice([1, 2, 6, 8]), _log(rng, 1, 8192)
    case = dict(op=op, tokens=tokens, top_k=top_k, experts=experts, skew=rng.choice([0.0, 1.1]))
    if op == "order":
        form = rng.choice(["dispatch", "dispatch backward", "combine", "combine backward"])
        kind = rng.choice(["bf16", "fp8", "f32"] if form == "dispatch" else ["bf16", "f32"])
        case.update(form=form, type=kind, hidden=16 * _log(rng, 1, 128) if kind == "fp8" else _log(rng, 16, 2048))
        return dict(case, add=rng.random() < 0.5) if form == "combine" else case
    if rng.random() < 0.3:
        case.update(experts=1, top_k=1, skew=0.0)
    form = rng.choice(["product", "product", "down"])
    n = _log(rng, 128, 2048) // 8 * 8 - (rng.randrange(1, 8) if rng.random() < 0.2 else 0)
    return dict(case, form=form, n=n, k=32 * _log(rng, 4, 64),
                out="bf16" if form == "down" else rng.choice(["bf16", "f32"]))


def _rows(case):
    return case["tokens"] * case["top_k"]


def _touched(case):
    """Experts that tokens reach (expectation under uniform routing)."""
    E, k = case["experts"], case["top_k"]
    return E * (1.0 - (1.0 - k / E) ** case["tokens"])


SIZE = {"none": 0, "bf16": 2, "f32": 4, "fp8": 1}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def work(case):
    if case["op"] == "norm":
        R, H, s = case["rows"], case["hidden"], SIZE[case["residual"]]
        if case["form"] == "backward":
            s = s or 2
            return {"bytes": R * H * (2 + s + s * case["past"] + s) + 4 * R + 6 * H, "flops": 9 * R * H}
        out = {"bf16": 2, "fp8": 1, "both": 3}[case["out"]]
        scales = 0 if case["out"] == "bf16" else 4 * R * -(-H // 128)
        return {"bytes": R * H * (2 + 2 * s + out) + scales + 4 * R + 2 * H, "flops": 5 * R * H}
    T, P = case["tokens"], _rows(case)
    if case["op"] == "order":
        H, s = case["hidden"], SIZE[case["type"]]
        if case["form"] == "dispatch":
            row = H * s + (4 * -(-H // 128) if case["type"] == "fp8" else 0)
            return {"bytes": (T + P) * row + 16 * P, "flops": 0}
        if case["form"] == "dispatch backward":
            return {"bytes": (T * 2 + P * s) * H + 12 * P, "flops": P * H}
        if case["form"] == "combine":
            return {"bytes": (T * s * (2 if case["add"] else 1) + P * 2) * H + 8 * P, "flops": 2 * P * H}
        return {"bytes": (T * s + 2 * P * 2) * H + 12 * P, "flops": 3 * P * H}
    N, K = case["n"], case["k"]
    given = 2 * P * K if case["form"] == "product" else 4 * P * K
    return {"bytes": given + _touched(case) * N * (K // 2 + K // 32) + (4 if case["out"] == "f32" else 2) * P * N,
            "flops": 2.0 * P * N * K}


# ---------------------------------------------------------------- inputs


def _routing(case, gen):
    """ids int64 [T, k] of top-k routing of random logits (plus a Zipf prior), and the routing weights."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if case["skew"]:
        prior = -case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        logits = logits + prior[torch.randperm(E, generator=gen, device="cuda")]
    top = logits.topk(k, dim=1)
    return top.indices, torch.softmax(top.values, 1)


def _order(ids, E):
    """slot int32 [P], pos int32 [T, k] and offs int32 [E + 1] of rows sorted by expert."""
    flat = ids.reshape(-1)
    slot = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(slot)
    pos[slot] = torch.arange(slot.numel(), device=slot.device)
    counts = torch.zeros(E, dtype=torch.int64, device=slot.device).scatter_add_(0, flat, torch.ones_like(flat))
    offs = torch.zeros(E + 1, dtype=torch.int32, device=slot.device)
    offs[1:] = counts.cumsum(0)
    return slot.int(), pos.view(ids.shape).int(), offs


def _scale_tiles(rows):
    """Scales [E, N, K / 32] as the product reads them: [E, ceil(N / 128), ceil(K / 128), 512], the bytes of a
    tile in the order (row % 32, row / 32, block)."""
    E, N, nb = rows.shape
    nt, kt = -(-N // 128), -(-nb // 4)
    t = torch.zeros((E, nt * 128, kt * 4), dtype=torch.uint8, device=rows.device)
    t[:, :N, :nb] = rows
    return t.view(E, nt, 4, 32, kt, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, nt, kt, 512).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
        return t if scale == 1.0 else t.mul_(scale)

    s = {"case": case}
    if case["op"] == "norm":
        R, H = case["rows"], case["hidden"]
        s["w"] = normal(H, scale=0.1) + (1.0 - case["offset"])
        kind = torch.float32 if case["residual"] == "f32" else torch.bfloat16
        if case["form"] == "forward":
            s["x"] = normal(R, H)
            s["r"] = normal(R, H, scale=3.0, dtype=kind) if case["residual"] != "none" else None
        else:
            s["total"] = normal(R, H, scale=3.0, dtype=kind)
            s["rstd"] = 1.0 / torch.sqrt((s["total"].float() ** 2).mean(1) + EPS)
            s["dy"] = normal(R, H, scale=0.05)
            s["past"] = normal(R, H, scale=0.05, dtype=kind) if case["past"] else None
        return s
    T, P, E = case["tokens"], _rows(case), case["experts"]
    ids, weights = _routing(case, gen)
    s["slot"], s["pos"], s["offs"] = _order(ids, E)
    s["weights"] = weights
    if case["op"] == "order":
        H = case["hidden"]
        if case["form"] == "dispatch":
            if case["type"] == "fp8":
                s["x"], s["scale"] = _quantized(normal(T, H).float())
            else:
                s["x"] = normal(T, H, dtype=TYPE[case["type"]])
        elif case["form"] == "dispatch backward":
            s["dxs"] = normal(P, H, scale=0.05, dtype=TYPE[case["type"]])
            s["drow"] = normal(P, dtype=torch.float32)
        else:
            s["y"] = normal(P, H)
            if case["form"] == "combine":
                s["add"] = normal(T, H, dtype=TYPE[case["type"]]) if case["add"] else None
            else:
                s["dout"] = normal(T, H, scale=0.05, dtype=TYPE[case["type"]])
        return s
    N, K = case["n"], case["k"]
    if case["form"] == "product":
        s["x"] = normal(P, K)
    else:
        s["gu"] = normal(P, 2 * K, scale=1.5)
    s["wq"] = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    mid = 126 - round(math.log2(3.0 * K ** 0.5))
    s["ws"] = torch.randint(mid - 1, mid + 2, (E, N, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    s["tiles"] = _scale_tiles(s["ws"])
    if E == 1:
        s["offs"] = None
    return s


# ---------------------------------------------------------------- plain forms


def _quantized(v):
    """e4m3 values [P, K] (as float8_e4m3fn) and scales [K / 128, P] of fp32 rows."""
    P, K = v.shape
    nb = -(-K // 128)
    b = torch.nn.functional.pad(v, (0, nb * 128 - K)).view(P, nb, 128)
    amax = b.abs().amax(dim=2)
    scale = (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=TINY)
    q = (b * (torch.ones_like(scale) / scale)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(P, nb * 128)[:, :K].to(torch.float8_e4m3fn).contiguous(), scale.t().contiguous()


def _plain_norm(case, s):
    w = s["w"].float() + case["offset"]
    if case["form"] == "backward":
        total, dy, rstd = s["total"].float(), s["dy"].float(), s["rstd"][:, None]
        n, g = total * rstd, dy * w
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if s["past"] is not None:
            dx = dx + s["past"].float()
        return [dx.to(s["total"].dtype), (dy * n).sum(0)]
    total = s["x"]
    if s["r"] is not None:
        total = (s["x"].float() + s["r"].float()).to(s["r"].dtype)
    t = total.float()
    rstd = 1.0 / torch.sqrt((t * t).mean(1) + EPS)
    y = t * rstd[:, None] * w
    out = [rstd] if s["r"] is None else [rstd, total]
    if case["out"] != "fp8":
        out.append(y.bfloat16())
    return out if case["out"] == "bf16" else out + list(_quantized(y))


def _plain_order(case, s):
    k, slot, pos = case["top_k"], s["slot"].long(), s["pos"].long()
    if case["form"] == "dispatch":
        token = slot // k
        back = torch.empty_like(slot)
        back[slot] = torch.arange(slot.numel(), device=slot.device)
        rows = s["x"].view(torch.uint8)[token].view(s["x"].dtype)
        scale = [s["scale"][:, token]] if case["type"] == "fp8" else []
        return [rows, *scale, s["weights"].reshape(-1)[slot], back.view(pos.shape).int()]
    if case["form"] == "dispatch backward":
        return [s["dxs"].float()[pos].sum(1).bfloat16(), s["drow"][pos]]
    if case["form"] == "combine":
        out = (s["y"].float()[pos] * s["weights"][:, :, None]).sum(1)
        if s["add"] is not None:
            out = out + s["add"].float()
        return out.to(TYPE[case["type"]])
    dout, y = s["dout"].float(), s["y"].float()
    token = slot // k
    dy = dout[token] * s["weights"].reshape(-1)[slot][:, None]
    return [dy.bfloat16(), (dout[token] * y).sum(1)[pos]]


def _e2m1(v):
    """Nearest e2m1 value, ties to the even code."""
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=6.0)


def _quantized4(v):
    """The values that fp32 rows [P, K] have in MXFP4: a block of 32 is scaled by the smallest power of two
    that brings it within +-6."""
    b = v.view(v.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(dim=2, keepdim=True))
    scale = torch.ldexp(torch.ones_like(m), (e - 2 - (m <= 0.75).int()).clamp(min=-127))
    return (_e2m1(b / scale) * scale).view(v.shape)


def _decoded(codes, scales):
    """fp32 values of packed codes [..., K / 2] (even elements in the low halves) and scales [..., K / 32]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return v * torch.exp2(scales.float() - 127.0).repeat_interleave(32, -1)


def _blocks(offs, P, E):
    """The rows of every expert in blocks of BLOCK: expert of each block [B], row numbers [B, BLOCK]
    and which of them are the expert's own. B is a bound that P and E give."""
    offs = offs.long()
    per = (offs[1:] - offs[:-1] + BLOCK - 1) // BLOCK
    ends = per.cumsum(0)
    b = torch.arange(P // BLOCK + min(E, P), device=offs.device)
    e = torch.searchsorted(ends, b, right=True).clamp(max=E - 1)
    first = offs[e] + (b - (ends - per)[e]) * BLOCK
    rows = first[:, None] + torch.arange(BLOCK, device=offs.device)
    mine = (rows < offs[e + 1][:, None]) & (b < ends[-1])[:, None]
    return e, rows.clamp(0, P - 1), mine


def _plain_mxfp4(case, s):
    P, E, N, K = _rows(case), case["experts"], case["n"], case["k"]
    if case["form"] == "product":
        x = _quantized4(s["x"].float())
    else:
        g, u = s["gu"].float().split(K, dim=1)
        x = _quantized4(g / (1.0 + torch.exp(-g)) * u)
    if E == 1:
        return (x @ _decoded(s["wq"][0], s["ws"][0]).t()).to(TYPE[case["out"]])
    e, rows, mine = _blocks(s["offs"], P, E)
    xb = torch.where(mine[:, :, None], x[rows], 0.0)
    few = e.numel() < E  # decode the weights of every block, or of every expert, whichever are fewer
    w = _decoded(s["wq"][e], s["ws"][e]) if few else _decoded(s["wq"], s["ws"])[e]
    yb = torch.bmm(xb, w.transpose(1, 2))
    y = torch.zeros((P + 1, N), device=yb.device)
    y[torch.where(mine, rows, P).reshape(-1)] = yb.reshape(-1, N)
    return y[:P].to(TYPE[case["out"]])


# ---------------------------------------------------------------- the library's calls


def _empty(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _own_norm(ft, case, s):
    R, H = case["rows"], case["hidden"]
    if case["form"] == "backward":
        dx, dw = torch.empty_like(s["total"]), _empty(H, dtype=torch.float32)
        ws = _empty(ft.ft_moe_rmsnorm_workspace_size(R, H), dtype=torch.uint8)
        ft.ft_moe_rmsnorm_backward(s["dy"], s["total"], s["w"], s["rstd"], dx, ws, dw=dw, dtotal=s["past"],
                                   weight_offset=case["offset"])
        return [dx, dw]
    out = {"rstd": _empty(R, dtype=torch.float32)}
    if s["r"] is not None:
        out["total"] = torch.empty_like(s["r"])
    if case["out"] != "fp8":
        out["y"] = _empty(R, H, dtype=torch.bfloat16)
    if case["out"] != "bf16":
        out["codes"] = _empty(R, H, dtype=torch.float8_e4m3fn)
        out["scales"] = _empty(-(-H // 128), R, dtype=torch.float32)
    ft.ft_moe_rmsnorm(s["x"], s["w"], EPS, residual=s["r"], weight_offset=case["offset"], **out)
    return list(out.values())


def _own_order(ft, case, s):
    T, k, P, H = case["tokens"], case["top_k"], _rows(case), case["hidden"]
    if case["form"] == "dispatch":
        xs, row_w, pos = _empty(P, H, dtype=s["x"].dtype), _empty(P, dtype=torch.float32), _empty(T, k, dtype=torch.int32)
        scale = _empty(-(-H // 128), P, dtype=torch.float32) if case["type"] == "fp8" else None
        ft.ft_moe_dispatch(s["x"], s["slot"], k, xs, x_scale=s.get("scale"), out_scale=scale, w=s["weights"], row_w=row_w,
                           pos=pos)
        return [t for t in (xs, scale, row_w, pos) if t is not None]
    if case["form"] == "dispatch backward":
        dx, dw = _empty(T, H, dtype=torch.bfloat16), _empty(T, k, dtype=torch.float32)
        ft.ft_moe_dispatch_backward(s["dxs"], s["pos"], dx, drow_w=s["drow"], dw=dw)
        return [dx, dw]
    if case["form"] == "combine":
        out = _empty(T, H, dtype=TYPE[case["type"]])
        ft.ft_moe_combine(s["y"], s["pos"], s["weights"], out, add=s["add"])
        return out
    dy, dw = _empty(P, H, dtype=torch.bfloat16), _empty(T, k, dtype=torch.float32)
    ft.ft_moe_combine_backward(s["dout"], s["y"], s["pos"], s["weights"], dy, dw=dw)
    return [dy, dw]


def _own_mxfp4(ft, case, s):
    P, E, N, K = _rows(case), case["experts"], case["n"], case["k"]
    codes, scales = _empty(P, K // 2, dtype=torch.uint8), ft.alloc_mxfp4_scales(P, K)
    if case["form"] == "product":
        ft.ft_moe_quantize_mxfp4(s["x"], codes, scales)
    else:
        ft.ft_moe_swiglu_quantize_mxfp4(s["gu"], None, codes, scales)
    ws = _empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8)
    y = _empty(P, N, dtype=TYPE[case["out"]])
    ft.ft_moe_group_gemm_mxfp4(codes, scales, s["wq"], s["tiles"], s["offs"], y, ws)
    return y


def run(state):
    case = state["case"]
    if own:
        import nvfp4_quantized_moe_gb300 as ft
        return {"norm": _own_norm, "order": _own_order, "mxfp4": _own_mxfp4}[case["op"]](ft, case, state)
    return {"norm": _plain_norm, "order": _plain_order, "mxfp4": _plain_mxfp4}[case["op"]](case, state)


# ---------------------------------------------------------------- 64 bits


def _nearest64(v, digits, lowest, most):
    """Nearest value with `digits` bits after the leading one, exponents from `lowest`, at most `most` (ties to even)."""
    a = v.abs().clamp(max=most)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** lowest))) - digits)
    return torch.copysign(torch.round(a / step).mul(step).clamp(max=most), v)


def _e4m3_64(y):
    codes, scales = torch.empty_like(y), []
    for at in range(0, y.shape[1], 128):
        part = y[:, at:at + 128]
        scale = (part.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
        codes[:, at:at + 128] = _nearest64(part / scale[:, None], 3, -6, E4M3_MAX)
        scales.append(scale)
    return codes, torch.stack(scales)


def _mxfp4_64(v):
    out = torch.empty_like(v)
    for at in range(0, v.shape[1], 32):
        part = v[:, at:at + 32]
        scale = torch.exp2(torch.ceil(torch.log2((part.abs().amax(1) / 6.0).clamp(min=2.0 ** -127))))[:, None]
        out[:, at:at + 32] = _nearest64(part / scale, 1, 0, 6.0) * scale
    return out


def _exact_norm(case, s):
    w = s["w"].double() + case["offset"]
    if case["form"] == "backward":
        total, dy = s["total"].double(), s["dy"].double()
        rstd = s["rstd"].double()[:, None]
        c = (dy * w * total).sum(1, keepdim=True) * rstd / case["hidden"]
        dx = rstd * dy * w - total * rstd * rstd * c
        return [dx if s["past"] is None else dx + s["past"].double(), (dy * (total * rstd)).sum(0)]
    total = s["x"].double()
    stored = []
    if s["r"] is not None:
        total = total + s["r"].double()
        stored = [total]
        total = total.to(s["r"].dtype).double()  # the norm is that of the sum as it is stored
    rstd = (total.pow(2).sum(1) / case["hidden"] + EPS).rsqrt()
    y = total * rstd[:, None] * w
    out = [rstd, *stored]
    if case["out"] != "fp8":
        out.append(y)
    return out if case["out"] == "bf16" else out + list(_e4m3_64(y))


def _exact_order(case, s):
    T, k, pos = case["tokens"], case["top_k"], s["pos"].long()
    if case["form"] == "dispatch":
        flat = pos.reshape(-1)
        rows = torch.empty((flat.numel(), case["hidden"]), dtype=torch.float64, device="cuda")
        rows[flat] = s["x"].double().repeat_interleave(k, 0)
        row_w = torch.empty(flat.numel(), dtype=torch.float64, device="cuda")
        row_w[flat] = s["weights"].double().reshape(-1)
        out = [rows]
        if case["type"] == "fp8":
            scale = torch.empty((s["scale"].shape[0], flat.numel()), dtype=torch.float64, device="cuda")
            scale[:, flat] = s["scale"].double().repeat_interleave(k, 1)
            out.append(scale)
        return out + [row_w, s["pos"]]
    total = torch.zeros((T, case["hidden"]), dtype=torch.float64, device="cuda")
    if case["form"] == "dispatch backward":
        for j in range(k):
            total += s["dxs"][pos[:, j]].double()
        return [total, s["drow"].double()[pos]]
    if case["form"] == "combine":
        for j in range(k):
            total += s["weights"][:, j, None].double() * s["y"][pos[:, j]].double()
        return total if s["add"] is None else total + s["add"].double()
    dout = s["dout"].double()
    dy = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.empty((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        dy[pos[:, j]] = s["weights"][:, j, None].double() * dout
        dw[:, j] = torch.einsum("th,th->t", dout, s["y"][pos[:, j]].double())
    return [dy, dw]


def _exact_mxfp4(case, s):
    P, E, N, K = _rows(case), case["experts"], case["n"], case["k"]
    if case["form"] == "product":
        x = _mxfp4_64(s["x"].double())
    else:
        g, u = s["gu"].double().chunk(2, dim=1)
        x = _mxfp4_64(g * u / (1.0 + torch.exp(-g)))
    at = [0, P] if s["offs"] is None else s["offs"].tolist()
    out = torch.zeros((P, N), dtype=torch.float64, device="cuda")
    for e in range(E):
        if at[e] == at[e + 1]:
            continue
        w = torch.empty((N, K), dtype=torch.float64, device="cuda")
        for half in (0, 1):
            c = (s["wq"][e] >> (4 * half)).int() & 15
            m, x2, sign = (c & 1).double(), (c >> 1) & 3, 1.0 - 2.0 * (c >> 3).double()
            w[:, half::2] = sign * torch.where(x2 == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(x2.double() - 1.0))
        w = (w.view(N, -1, 32) * torch.exp2(s["ws"][e].double() - 127.0)[:, :, None]).view(N, K)
        out[at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ w.t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "order": _exact_order, "mxfp4": _exact_mxfp4}[case["op"]](case, s)
