"""SwiGLU of gates far from zero: the sigmoid keeps its relative accuracy down to where fp32 ends.

The fast exponential is within 2 + 1.173 |g| units of 2^-23 (CUDA's documented bound), 1.3e-5
at |g| = 88; sigmoid, products and the formula add a few units more: 2^-15 in all, and the store 2^-8.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
REL = 2.0 ** -15


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _rows(lo, hi, up):
    g = torch.linspace(lo, hi, 512, dtype=torch.float64).bfloat16().view(4, 128)
    return torch.cat([g, torch.full_like(g, up)], 1).cuda()


# the sigmoid of -88.5 is 3.7e-39, below fp32's smallest normal number; `up` brings the product back
RANGES = [(-88.5, -80.0, 2.0 ** 60), (-80.0, -8.0, 2.0 ** 20), (-8.0, 8.0, 1.5), (8.0, 88.5, 0.75)]


@pytest.mark.parametrize("lo,hi,up", RANGES)
def test_forward(ft, lo, hi, up):
    gu = _rows(lo, hi, up)
    h = torch.empty((4, 128), dtype=torch.bfloat16, device="cuda")
    ft.ft_moe_swiglu(gu, None, h)
    g, u = gu.double().chunk(2, 1)
    ref = g * torch.sigmoid(g) * u
    assert ((h.double() - ref).abs() <= (2.0 ** -8 + REL) * ref.abs()).all()


@pytest.mark.parametrize("lo,hi,up", RANGES)
def test_backward(ft, lo, hi, up):
    gu = _rows(lo, hi, up)
    dh = torch.full((4, 128), up, dtype=torch.bfloat16, device="cuda")
    dgu, w, dw = torch.empty_like(gu), torch.full((4,), 0.5, device="cuda"), torch.empty(4, device="cuda")
    ft.ft_moe_swiglu_backward(gu, w, dh, dgu, dw)
    g, u = gu.double().chunk(2, 1)
    s, d = torch.sigmoid(g), dh.double()
    slope, silu = s * (1 + g * torch.sigmoid(-g)), g * s
    dg, du = 0.5 * d * u * slope, 0.5 * d * silu
    # the two terms of the slope cancel near g = -1.28: each is within REL
    terms = 0.5 * d * u * s * (1 + g.abs() * torch.sigmoid(-g))
    assert ((dgu[:, :128].double() - dg).abs() <= 2.0 ** -8 * dg.abs() + REL * terms).all()
    assert ((dgu[:, 128:].double() - du).abs() <= (2.0 ** -8 + REL) * du.abs()).all()
    assert ((dw.double() - (d * silu * u).sum(1)).abs() <= REL * (d * silu * u).abs().sum(1)).all()


@pytest.mark.parametrize("lo,hi,up", RANGES)
def test_in_8_bits(ft, lo, hi, up):
    gu = _rows(lo, hi, up)
    codes, scales = torch.empty((4, 128), dtype=torch.uint8, device="cuda"), torch.empty((1, 4), device="cuda")
    ft.ft_moe_swiglu_quantize_fp8(gu, None, codes, scales)
    g, u = gu.double().chunk(2, 1)
    ref = g * torch.sigmoid(g) * u
    scale = ref.abs().amax(1) / 448
    assert ((scales[0].double() - scale).abs() <= REL * scale).all()
    value = codes.view(torch.float8_e4m3fn).double() * scales[0, :, None].double()
    # half an e4m3 step: 2^-4 of the value, or 2^-10 of the scale below the smallest normal code
    assert ((value - ref).abs() <= (2.0 ** -4 + REL) * ref.abs() + 2.0 ** -10 * 1.001 * scale[:, None]).all()
