"""Measured cases of the expert products: the grouped bf16 products of ragged expert batches
with their gradients, the 8-bit floating-point products with a scale per block of 128, and the
SwiGLU step between the two products of an expert.

Each case has a plain form (elementary torch operations in fp32, rounded once at the end) and
the library's own calls; ``own`` chooses between them. Layer sizes are those of the layer
families in ``synth.SHAPES`` (qwen36, dsv4, odd_h).

Rows of all experts lie one after the other, sorted by expert: expert e owns the rows
[offs[e], offs[e + 1]) of x, y, dx and dy, which is the order ``ft_moe_align`` gives with
block = 1.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest block scale
BLOCK = 64          # rows per batch entry of the plain products


def listed():
    return [
        # one token, top-8 of 256: the down product of a single-token step, 8 experts with a row each
        dict(name="down 1 token", op="product", form="forward", tokens=1, top_k=8, experts=256, n=2048, k=512,
             skew=0.0, out="bf16"),
        # an ordinary decode batch: gate_up of 64 tokens, most experts touched with one to six rows
        dict(name="gate_up 64 tokens", op="product", form="forward", tokens=64, top_k=8, experts=256, n=1024,
             k=2048, skew=0.0, out="bf16"),
        # prefill / training forward: skewed routing, groups from a few rows to thousands
        dict(name="gate_up 8192 tokens", op="product", form="forward", tokens=8192, top_k=8, experts=256, n=1024,
             k=2048, skew=1.1, out="bf16"),
        # gradient of the inputs, an odd number of tokens, widths that are no multiple of 256, fp32 out
        dict(name="down dgrad 1999 tokens", op="product", form="dgrad", tokens=1999, top_k=8, experts=128, n=640,
             k=512, skew=1.1, out="f32"),
        # gradient of the inputs of a wide layer: 8.6 GB of weights, the largest case
        dict(name="wide dgrad 4096 tokens", op="product", form="dgrad", tokens=4096, top_k=8, experts=256, n=4096,
             k=4096, skew=1.1, out="bf16"),
        # gradient of the weights into fp32 (what an optimiser accumulates)
        dict(name="gate_up wgrad 8192 tokens", op="product", form="wgrad", tokens=8192, top_k=8, experts=256,
             n=1024, k=2048, skew=1.1, out="f32"),
        # the shared expert of one token in 8 bits: two small launches, latency
        dict(name="fp8 shared 1 token", op="fp8", tokens=1, top_k=1, experts=1, n=1024, k=2048, skew=0.0, out="bf16"),
        # decode batch over 8-bit experts
        dict(name="fp8 gate_up 64 tokens", op="fp8", tokens=64, top_k=8, experts=256, n=1024, k=2048, skew=0.0,
             out="bf16"),
        # prefill over 8-bit experts, skewed
        dict(name="fp8 gate_up 8192 tokens", op="fp8", tokens=8192, top_k=8, experts=256, n=1024, k=2048, skew=1.1,
             out="bf16"),
        # the plain 8-bit product: the wide layer's shared expert over a prefill chunk
        dict(name="fp8 shared 4096 tokens", op="fp8", tokens=4096, top_k=1, experts=1, n=4096, k=4096, skew=0.0,
             out="bf16"),
        # between the two 8-bit products of a decode batch: SwiGLU whose result is stored in 8 bits
        dict(name="swiglu fp8 64 tokens", op="swiglu", form="quantize", rows=512, inter=512, weighted=False),
        # backward of the weighted SwiGLU of a training step
        dict(name="swiglu backward 8192 tokens", op="swiglu", form="backward", rows=65536, inter=512, weighted=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "dgrad", "wgrad", "fp8", "fp8 dense", "swiglu"])
    if kind == "swiglu":
        form = rng.choice(["forward", "backward", "quantize"])
        inter = 16 * _log(rng, 1, 128) if form == "quantize" else _log(rng, 16, 2048)
        return dict(op="swiglu", form=form, rows=_log(rng, 1, 65536), inter=inter, weighted=rng.random() < 0.5)
    experts = 1 if kind == "fp8 dense" else rng.choice([8, 60, 128, 256])
    top_k = 1 if experts == 1 else rng.choice([1, 2, 6, 8])
    tokens = _log(rng, 1, 8192)
    unit = 16 if kind.startswith("fp8") else 8
    n, k = unit * _log(rng, 128 // unit, 2048 // unit), unit * _log(rng, 128 // unit, 2048 // unit)
    if kind.startswith("fp8") and rng.random() < 0.3:
        n -= rng.randrange(1, 16)
    case = dict(op="fp8" if kind.startswith("fp8") else "product", tokens=tokens, top_k=top_k, experts=experts, n=n,
                k=k, skew=rng.choice([0.0, 1.1]) if experts > 1 else 0.0, out=rng.choice(["bf16", "bf16", "f32"]))
    if not kind.startswith("fp8"):
        case["form"] = kind
    return case


def _rows(case):
    return case["tokens"] * case["top_k"]


def _touched(case):
    """Experts that tokens reach (expectation under uniform routing)."""
    E, k = case["experts"], case["top_k"]
    return E * (1.0 - (1.0 - k / E) ** case["tokens"])


def work(case):
    if case["op"] == "swiglu":
        P, I = case["rows"], case["inter"]
        blocks = -(-I // 128)
        w = 4 * P if case["weighted"] else 0
        moved = {"forward": 4 * I + 2 * I, "backward": 4 * I + 2 * I + 4 * I, "quantize": 4 * I + I + 4 * blocks}
        extra = 2 * w if case["form"] == "backward" else w
        return {"bytes": P * moved[case["form"]] + extra, "flops": P * I * (20 if case["form"] == "backward" else 8)}
    P, N, K, E = _rows(case), case["n"], case["k"], case["experts"]
    ob = 4 if case["out"] == "f32" else 2
    flops = 2.0 * P * N * K
    if case["op"] == "fp8":
        scales = 4.0 * (-(-N // 128)) * (-(-K // 128))
        return {"bytes": 2 * P * K + _touched(case) * (N * K + scales) + ob * P * N, "flops": flops}
    if case["form"] == "wgrad":
        return {"bytes": 2 * P * (N + K) + ob * E * N * K, "flops": flops}
    rows = 2 * P * K + ob * P * N if case["form"] == "forward" else 2 * P * N + ob * P * K
    return {"bytes": rows + 2 * _touched(case) * N * K, "flops": flops}


# ---------------------------------------------------------------- inputs


def _offsets(case, gen):
    """Expert offsets int32 [E + 1] of top-k routing of random logits (plus a Zipf prior)."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if case["skew"]:
        prior = -case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        logits = logits + prior[torch.randperm(E, generator=gen, device="cuda")]
    ids = logits.topk(k, dim=1).indices.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, ids, torch.ones_like(ids))
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[1:] = counts.cumsum(0)
    return offs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        return t if scale == 1.0 else t.mul_(scale)

    if case["op"] == "swiglu":
        P, I = case["rows"], case["inter"]
        s = {"case": case, "gu": normal(P, 2 * I, scale=1.5), "w": None}
        if case["weighted"]:  # routing weights of the rows
            s["w"] = torch.rand(P, generator=gen, device="cuda") * 0.5
        if case["form"] == "backward":
            s["dh"] = normal(P, I, scale=0.05)
        return s
    P, N, K, E = _rows(case), case["n"], case["k"], case["experts"]
    s = {"case": case, "offs": _offsets(case, gen) if E > 1 else None}
    if case["op"] == "fp8":
        s["x"] = normal(P, K)
        s["wq"] = normal(E, N, K, scale=32.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        shape = (E, -(-N // 128), -(-K // 128))
        s["ws"] = (torch.rand(shape, generator=gen, device="cuda") + 0.5) * 2.0 ** -8
    else:
        if case["form"] != "dgrad":
            s["x"] = normal(P, K)
        if case["form"] != "forward":
            s["dy"] = normal(P, N, scale=0.05)
        if case["form"] != "wgrad":
            s["w"] = normal(E, N, K, scale=K ** -0.5)
    return s


# ---------------------------------------------------------------- plain forms


def _out(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


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


def _take(a, rows, mine):
    """fp32 [B, BLOCK, columns] of the blocks' rows, zero where a block has no row."""
    return torch.where(mine[:, :, None], a[rows].float(), 0.0)


def _put(yb, rows, mine, P):
    y = torch.zeros((P + 1, yb.shape[2]), device=yb.device)
    y[torch.where(mine, rows, P).reshape(-1)] = yb.reshape(-1, yb.shape[2])
    return y[:P]


def _plain_product(case, s):
    P, E = _rows(case), case["experts"]
    e, rows, mine = _blocks(s["offs"], P, E)
    if case["form"] == "forward":
        y = torch.bmm(_take(s["x"], rows, mine), s["w"][e].float().transpose(1, 2))
        return _put(y, rows, mine, P).to(_out(case))
    dy = _take(s["dy"], rows, mine)
    if case["form"] == "dgrad":
        return _put(torch.bmm(dy, s["w"][e].float()), rows, mine, P).to(_out(case))
    dw = torch.zeros((E, case["n"], case["k"]), device=dy.device)
    dw.index_add_(0, e, torch.bmm(dy.transpose(1, 2), _take(s["x"], rows, mine)))
    return dw.to(_out(case))


def _quantized(v):
    """e4m3 values [P, K] (as float8_e4m3fn) and scales [K / 128, P] of fp32 rows."""
    P, K = v.shape
    nb = -(-K // 128)
    b = torch.nn.functional.pad(v, (0, nb * 128 - K)).view(P, nb, 128)
    amax = b.abs().amax(dim=2)
    scale = (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=TINY)
    q = (b * (torch.ones_like(scale) / scale)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(P, nb * 128)[:, :K].to(torch.float8_e4m3fn), scale.t().contiguous()


def _spread(scale, N, K):
    """Scales [..., ceil(N / 128), ceil(K / 128)] at every element [..., N, K]."""
    return scale.repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]


def _plain_fp8(case, s):
    P, N, K, E = _rows(case), case["n"], case["k"], case["experts"]
    q, scale = _quantized(s["x"].float())
    x = q.float() * scale.t().repeat_interleave(128, 1)[:, :K]
    wq = s["wq"].view(torch.float8_e4m3fn)
    if E == 1:
        return (x @ (wq[0].float() * _spread(s["ws"][0], N, K)).t()).to(_out(case))
    e, rows, mine = _blocks(s["offs"], P, E)
    w = s["wq"][e].view(torch.float8_e4m3fn).float() * _spread(s["ws"][e], N, K)
    return _put(torch.bmm(_take(x, rows, mine), w.transpose(1, 2)), rows, mine, P).to(_out(case))


def _plain_swiglu(case, s):
    I = case["inter"]
    g, u = s["gu"].float().split(I, dim=1)
    sig = 1.0 / (1.0 + torch.exp(-g))
    w = s["w"][:, None] if s["w"] is not None else torch.ones((), device=g.device)
    if case["form"] == "forward":
        return (w * (g * sig * u)).bfloat16()
    if case["form"] == "quantize":
        q, scale = _quantized(w * (g * sig * u))
        return [q, scale]
    dh = s["dh"].float()
    dg = w * dh * u * (sig * (1.0 + g * (1.0 - sig)))
    du = w * dh * (g * sig)
    dw = (dh * (g * sig * u)).sum(1) if s["w"] is not None else None
    return [torch.cat([dg, du], 1).bfloat16(), dw]


# ---------------------------------------------------------------- the library's calls


def _own_product(ft, case, s):
    P, N, K, E = _rows(case), case["n"], case["k"], case["experts"]
    ws = torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device="cuda")
    if case["form"] == "forward":
        y = torch.empty((P, N), dtype=_out(case), device="cuda")
        ft.ft_moe_group_gemm(s["x"], s["w"], s["offs"], y, ws)
        return y
    if case["form"] == "dgrad":
        dx = torch.empty((P, K), dtype=_out(case), device="cuda")
        ft.ft_moe_group_gemm_dgrad(s["dy"], s["w"], s["offs"], dx, ws)
        return dx
    dw = torch.empty((E, N, K), dtype=_out(case), device="cuda")
    ft.ft_moe_group_gemm_wgrad(s["dy"], s["x"], s["offs"], dw, ws)
    return dw


def _own_fp8(ft, case, s):
    P, N, K, E = _rows(case), case["n"], case["k"], case["experts"]
    codes = torch.empty((P, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((-(-K // 128), P), dtype=torch.float32, device="cuda")
    ws = torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device="cuda")
    y = torch.empty((P, N), dtype=_out(case), device="cuda")
    ft.ft_moe_quantize_fp8(s["x"], codes, scales)
    ft.ft_moe_group_gemm_fp8(codes, scales, s["wq"], s["ws"], s["offs"], y, ws)
    return y


def _own_swiglu(ft, case, s):
    P, I = case["rows"], case["inter"]
    if case["form"] == "forward":
        h = torch.empty((P, I), dtype=torch.bfloat16, device="cuda")
        ft.ft_moe_swiglu(s["gu"], s["w"], h)
        return h
    if case["form"] == "quantize":
        codes = torch.empty((P, I), dtype=torch.uint8, device="cuda")
        scales = torch.empty((-(-I // 128), P), dtype=torch.float32, device="cuda")
        ft.ft_moe_swiglu_quantize_fp8(s["gu"], s["w"], codes, scales)
        return [codes.view(torch.float8_e4m3fn), scales]
    dgu = torch.empty((P, 2 * I), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(P, dtype=torch.float32, device="cuda") if s["w"] is not None else None
    ft.ft_moe_swiglu_backward(s["gu"], s["w"], s["dh"], dgu, dw)
    return [dgu, dw]


def run(state):
    case = state["case"]
    if own:
        import nvfp4_quantized_moe_gb300 as ft
        return {"product": _own_product, "fp8": _own_fp8, "swiglu": _own_swiglu}[case["op"]](ft, case, state)
    return {"product": _plain_product, "fp8": _plain_fp8, "swiglu": _plain_swiglu}[case["op"]](case, state)


# ---------------------------------------------------------------- 64 bits


def _e4m3_64(v):
    """Nearest e4m3 value (ties to the even mantissa, saturating) of fp64 numbers."""
    m = v.abs().clamp(max=E4M3_MAX)
    exponent = torch.floor(torch.log2(m.clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3.0)
    return torch.sign(v) * torch.round(m / step).mul(step).clamp(max=E4M3_MAX)


def _quantized_64(v):
    codes, scales = torch.empty_like(v), []
    for at in range(0, v.shape[1], 128):
        part = v[:, at:at + 128]
        scale = (part.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
        codes[:, at:at + 128] = _e4m3_64(part / scale[:, None])
        scales.append(scale)
    return codes, torch.stack(scales)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "swiglu":
        g, u = s["gu"].double().chunk(2, dim=1)
        w = torch.ones(g.shape[0], device="cuda", dtype=torch.float64) if s["w"] is None else s["w"].double()
        silu = g / (1.0 + torch.exp(-g))
        if case["form"] == "forward":
            return w[:, None] * silu * u
        if case["form"] == "quantize":
            return list(_quantized_64(w[:, None] * silu * u))
        dh = s["dh"].double()
        slope = silu / g + silu * (1.0 - silu / g)
        slope = torch.where(g == 0, 0.5, slope)
        dgu = torch.cat([w[:, None] * dh * u * slope, w[:, None] * dh * silu], 1)
        return [dgu, None if s["w"] is None else (dh * silu * u).sum(1)]
    P, N, K, E = _rows(case), case["n"], case["k"], case["experts"]
    at = [0, P] if s["offs"] is None else s["offs"].tolist()
    if case["op"] == "product" and case["form"] == "wgrad":
        out = torch.empty((E, N, K), dtype=torch.float64, device="cuda")
        for e in range(E):
            torch.matmul(s["dy"][at[e]:at[e + 1]].double().t(), s["x"][at[e]:at[e + 1]].double(), out=out[e])
        return out
    if case["op"] == "fp8":
        codes, scales = _quantized_64(s["x"].double())
        for b in range(scales.shape[0]):
            codes[:, b * 128:(b + 1) * 128] *= scales[b][:, None]
        src, cols = codes, N
    else:
        src = (s["x"] if case["form"] == "forward" else s["dy"]).double()
        cols = N if case["form"] == "forward" else K
    out = torch.zeros((P, cols), dtype=torch.float64, device="cuda")
    for e in range(E):
        if at[e] == at[e + 1]:
            continue
        if case["op"] == "fp8":
            w = s["wq"][e].view(torch.float8_e4m3fn).double()
            scale = s["ws"][e].double()
            for b in range(scale.shape[0]):
                for c in range(scale.shape[1]):
                    w[b * 128:(b + 1) * 128, c * 128:(c + 1) * 128] *= scale[b, c]
        else:
            w = s["w"][e].double()
        rows = src[at[e]:at[e + 1]]
        out[at[e]:at[e + 1]] = rows @ w if case["op"] == "product" and case["form"] == "dgrad" else rows @ w.t()
    return out
