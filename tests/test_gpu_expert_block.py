"""The residual norm, the tokens' sorting and the products together, as a layer runs them (examples/expert_layer.py): a
residual block's training step against torch's autograd in 64 bits, and the 4-bit serving step against the same
arithmetic on the values that its codes stand for."""
import importlib.util
import os

import pytest
import torch

from mxfp4_cases import decode, row_scales, rule

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 64, 8, 2), (37, 264, 64, 8, 2), (300, 128, 72, 16, 4), (700, 640, 512, 8, 2)])
def test_training_block_matches_autograd(layer, T, H, I, E, k, kind):
    """Output and every gradient within a few bf16 roundings (2^-8 at most) of the 64-bit ones: total and y, gu, h, dh,
    dgu, dy and dx are rounded to bf16 on the way: 6 * 2^-8 = 2.4e-2 in norm, if all were the worst at once."""
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda") * s[-1] ** -0.5  # noqa: E731
    x = (mk(T, H) * H ** 0.5).bfloat16().requires_grad_()
    r = (mk(T, H) * H ** 0.5).to(kind).requires_grad_()
    wn = (1 + 0.3 * torch.randn(H, generator=gen, device="cuda")).requires_grad_()
    w = [mk(E, H).requires_grad_(), mk(E, 2 * I, H).bfloat16().requires_grad_(), mk(E, H, I).bfloat16().requires_grad_()]
    dout, dstream = torch.randn((T, H), generator=gen, device="cuda"), torch.randn((T, H), generator=gen, device="cuda").to(kind)
    out, total = layer.train_block(x, r, wn, *w, k)
    got = torch.autograd.grad((out * dout).sum() + (total.float() * dstream.float()).sum(), [x, r, wn, *w])

    leaves = [a.detach().double().requires_grad_() for a in (x, r, wn, *w)]
    x64, r64, wn64, rt64, gu64, dn64 = leaves
    t64 = x64 + r64
    stored = t64 + (total.detach().double() - t64.detach())  # the norm is that of the stored sum
    y64 = stored * (stored.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * wn64
    logits = y64 @ rt64.t()
    yb = y64.detach().float().bfloat16()
    ids, _ = layer.route((yb.float() @ w[0].detach().t()).contiguous(), k)
    kept = torch.softmax(logits, 1).gather(1, ids.long())
    weights = kept / kept.sum(1, keepdim=True)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            g, u = (y64[t] @ gu64[e].t()).chunk(2, dim=1)
            ref = ref.index_add(0, t, weights[t, j, None] * (torch.nn.functional.silu(g) * u) @ dn64[e].t())
    want = torch.autograd.grad((ref * dout.double()).sum() + (t64 * dstream.double()).sum(), leaves)
    assert _rel(out.detach(), ref.detach()) <= 2.4e-2
    for a, b in zip(got, want):
        assert _rel(a, b) <= 2.4e-2


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 64, 8, 2), (50, 640, 96, 8, 4), (900, 512, 544, 4, 2), (3000, 1024, 512, 8, 2)])
def test_4_bit_serving_step(layer, T, H, I, E, k):
    """Against 64-bit arithmetic on the decoded weights, tokens quantized by the rule. What is not exact: gu is rounded to
    bf16 (2^-8), so that h and with it some codes of h come out a step away (a step is at most a third of a value, and
    falls to the other side where h lies within 2^-8 of a border, one in 64 values: 0.33 / 8 = 4% in norm); y is rounded to bf16."""
    ft = layer.ft
    gen = torch.Generator(device="cuda").manual_seed(T)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda") * s[-1] ** -0.5  # noqa: E731

    def weights(w):
        e, n, kk = w.shape
        codes = torch.empty((e, n, kk // 2), dtype=U8, device="cuda")
        tiles = torch.empty((e, (n + 127) // 128, (kk + 127) // 128, 512), dtype=U8, device="cuda")
        ft.ft_moe_quantize_mxfp4_weights(w, codes, tiles)
        c, s = rule(w.view(e * n, kk).float())
        return codes, tiles, decode(codes, s.view(e, n, -1))

    gu, gut, gu64 = weights(mk(E, 2 * I, H))
    dn, dnt, dn64 = weights(mk(E, H, I).bfloat16())
    x = (mk(T, H) * H ** 0.5).bfloat16()
    ids, w = layer.route(torch.randn((T, E), generator=gen, device="cuda"), k)
    shared = torch.randn((T, H), generator=gen, device="cuda")
    out = layer.serve_forward_mxfp4(x, ids, w, gu, gut, dn, dnt, shared=shared)
    codes, scales = torch.empty((T, H // 2), dtype=U8, device="cuda"), ft.alloc_mxfp4_scales(T, H)
    ft.ft_moe_quantize_mxfp4(x, codes, scales)
    x64 = decode(codes, row_scales(scales, H))
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            g, u = (x64[t] @ gu64[e].t()).chunk(2, dim=1)
            h = (torch.nn.functional.silu(g) * u).float()
            c, s = rule(h)
            packed = (c[:, 0::2] | (c[:, 1::2] << 4)).to(U8)
            ref.index_add_(0, t, w[t, j, None].double() * (decode(packed, s) @ dn64[e].t()))
    assert _rel(out.double() - shared.double(), ref) <= 6e-2


def test_norm_feeds_the_8_bit_product(layer):
    """The norm's 8-bit output goes into dispatch and product as it is: the same as quantizing the fp32 norm."""
    ft = layer.ft
    T, H, N, E, k = 130, 512, 256, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    w = (torch.randn((E, N, H), generator=gen, device="cuda") * 16).to(torch.float8_e4m3fn)
    wsc = torch.rand((E, N // 128, H // 128), generator=gen, device="cuda") + 0.5
    norm = torch.ones(H, device="cuda")
    ids = torch.rand((T, E), generator=gen, device="cuda").topk(k, 1).indices.int()
    plan = layer.Plan(ids, E)
    codes, scales = torch.empty((T, H), dtype=U8, device="cuda"), torch.empty((H // 128, T), device="cuda")
    ft.ft_moe_rmsnorm(x, norm, 1e-6, codes=codes, scales=scales)
    xc, xs = torch.empty((T * k, H), dtype=U8, device="cuda"), torch.empty((H // 128, T * k), device="cuda")
    ft.ft_moe_dispatch(codes, plan.slot, k, xc, x_scale=scales, out_scale=xs)
    y, ws = torch.empty((T * k, N), device="cuda"), torch.empty(256, dtype=U8, device="cuda")
    ft.ft_moe_group_gemm_fp8(xc, xs, w, wsc, plan.offs, y, ws)
    assert ft.ft_moe_read_status(ws) == 0
    t = x.double()
    n64 = t * (t.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()
    rows = n64[plan.slot.long() // k]
    e_of = torch.bucketize(torch.arange(T * k, device="cuda"), plan.offs[1:].long(), right=True)
    w64 = w.double() * wsc.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    ref = torch.einsum("ph,pnh->pn", rows, w64[e_of])
    # e4m3: half a step is 2^-4 of a value at most, 2^-5.3 in norm for smoothly distributed ones
    assert _rel(y, ref) <= 4e-2
