"""The 8-bit row quantizer and the SwiGLU kernels, through the C ABI.

The quantizer is compared bit for bit with its rule in correctly rounded fp32 (on the CPU).
SwiGLU is compared with the formulas in 64 bits: the fast exponential and division are within a few
1e-7 (2^-20 is allowed), the store rounds to 2^-8 relative.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _rule(v):
    """Codes and scales of fp32 rows (CPU: every operation correctly rounded)."""
    P, K = v.shape
    nb = -(-K // 128)
    b = torch.nn.functional.pad(v, (0, nb * 128 - K)).view(P, nb, 128)
    scale = (b.abs().amax(2) / torch.tensor(448.0)).clamp(min=2.0 ** -126)
    q = (b * (1.0 / scale)[:, :, None]).view(P, nb * 128)[:, :K]
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale.t()


def _quantize(ft, x, pad=0):
    P, K = x.shape
    codes = torch.full((P, K + 16 * pad), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-K // 128), P + pad), -1.0, device="cuda")
    ft.ft_moe_quantize_fp8(x, codes[:, :K], scales[:, :P])
    if pad:
        assert (codes[:, K:] == 0xAA).all() and (scales[:, P:] == -1).all()
    return codes[:, :K], scales[:, :P]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("P,K", [(1, 16), (1, 2048), (3, 128), (17, 144), (100, 2000), (33, 4096), (5000, 256)])
def test_quantizer_is_bit_exact(ft, P, K, dtype):
    gen = torch.Generator().manual_seed(P + K)
    x = torch.randn((P, K), generator=gen) * torch.exp2(torch.randint(-40, 40, (P, 1), generator=gen).float())
    x = x.to(dtype)
    if P > 2:
        x[1] = 0
        x[2, :K // 2] = 0
    codes, scales = _quantize(ft, x.cuda(), pad=P % 3)
    ref_c, ref_s = _rule(x.float())
    assert torch.equal(scales.cpu(), ref_s)
    c = codes.cpu()
    same = (c == ref_c) | ((c & 0x7F == 0) & (ref_c & 0x7F == 0))
    assert same.all()


def test_quantizer_edges(ft):
    """Magnitudes near the fp32 limits; infinities and NaN make their block not finite, and no other."""
    x = torch.zeros((6, 256))
    x[0, 5] = 1e-44
    x[1, 0], x[1, 1] = 3.0e38, -3.3e38
    x[2, 130] = float("inf")
    x[3, 7] = float("nan")
    x[4, :] = torch.linspace(-1, 1, 256)
    x[5, 255] = -2.0 ** -126
    codes, scales = _quantize(ft, x.cuda())
    value = codes.view(torch.float8_e4m3fn).float() * scales.t().repeat_interleave(128, 1)
    assert torch.isfinite(value[[0, 1, 4, 5]]).all()
    assert torch.isfinite(value[2, :128]).all() and not torch.isfinite(value[2, 128:]).any()
    assert not torch.isfinite(value[3, :128]).any() and torch.isfinite(value[3, 128:]).all()
    ref_c, ref_s = _rule(x[[0, 1, 4, 5]])
    assert torch.equal(scales.cpu()[:, [0, 1, 4, 5]], ref_s)
    assert torch.equal(codes.cpu()[[0, 1, 4, 5]] & 0x7F, ref_c & 0x7F)


def _inputs(P, I, weighted, seed=0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    gu = (torch.randn((P, 2 * I + pad), generator=gen, device="cuda") * 2).bfloat16()[:, :2 * I]
    dh = torch.randn((P, I + pad), generator=gen, device="cuda").bfloat16()[:, :I]
    w = torch.rand(P, generator=gen, device="cuda") if weighted else None
    return gu, dh, w


def _formula(gu, w, dh=None):
    I = gu.shape[1] // 2
    g, u = gu[:, :I].double(), gu[:, I:].double()
    s = torch.sigmoid(g)
    wd = 1.0 if w is None else w.double()[:, None]
    h = wd * g * s * u
    if dh is None:
        return h
    d = dh.double()
    dg, du = wd * d * u * s * (1 + g * (1 - s)), wd * d * g * s
    return dg, du, (d * g * s * u).sum(1), (wd * d * u).abs() * (1 + g.abs()), (d * g * s * u).abs().sum(1)


# I: vector steps and their tails, odd widths (element loads); pad: rows that are not 16-byte aligned
CASES = [(1, 512, 0), (7, 8, 0), (33, 256, 0), (300, 520, 8), (5, 1, 0), (64, 333, 0), (40, 512, 3), (20, 2048, 0), (3000, 64, 0)]


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("P,I,pad", CASES)
def test_swiglu(ft, P, I, pad, weighted):
    gu, _, w = _inputs(P, I, weighted, pad=pad)
    h = torch.full((P, I + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    ft.ft_moe_swiglu(gu, w, h[:, :I])
    ref = _formula(gu, w)
    assert ((h[:, :I].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -19) * ref.abs() + 1e-38).all()
    assert (h[:, I:] == 7).all()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("P,I,pad", CASES)
def test_swiglu_backward(ft, P, I, pad, weighted):
    gu, dh, w = _inputs(P, I, weighted, seed=1, pad=pad)
    dgu = torch.full((P, 2 * I + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((P,), float("nan"), device="cuda")
    ft.ft_moe_swiglu_backward(gu, w, dh, dgu[:, :2 * I], dw)
    dg, du, dref, mag, wmag = _formula(gu, w, dh)
    for got, ref in ((dgu[:, :I], dg), (dgu[:, I:2 * I], du)):
        assert ((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag + 1e-38).all()
    assert (dgu[:, 2 * I:] == 7).all()
    assert ((dw.double() - dref).abs() <= (I + 8) * 2.0 ** -23 * wmag + 1e-38).all()
    again, dw2 = torch.empty((P, 2 * I), dtype=torch.bfloat16, device="cuda"), torch.empty(P, device="cuda")
    ft.ft_moe_swiglu_backward(gu, w, dh, again, dw2)
    assert torch.equal(again, dgu[:, :2 * I]) and torch.equal(dw2, dw)
    ft.ft_moe_swiglu_backward(gu, w, dh, again, None)
    assert torch.equal(again, dgu[:, :2 * I])


def test_swiglu_backward_matches_differences(ft):
    """Central differences of the forward formula in 64 bits (step 1e-4: error ~ step^2)."""
    P, I = 9, 40
    gu, dh, w = _inputs(P, I, True, seed=2)
    dgu, dw = torch.empty((P, 2 * I), dtype=torch.bfloat16, device="cuda"), torch.empty(P, device="cuda")
    ft.ft_moe_swiglu_backward(gu, w, dh, dgu, dw)
    h, g64, w64, d = 1e-4, gu.double(), w.double(), dh.double()

    def loss(a, b):  # per row
        s = torch.sigmoid(a[:, :I])
        return (d * b[:, None] * a[:, :I] * s * a[:, I:]).sum(1)

    diff = torch.empty((P, 2 * I), dtype=torch.float64, device="cuda")
    for c in range(2 * I):
        step = torch.zeros_like(g64)
        step[:, c] = h
        diff[:, c] = (loss(g64 + step, w64) - loss(g64 - step, w64)) / (2 * h)
    scale = (d.abs().max() * gu.double().abs().max())
    assert ((dgu.double() - diff).abs() <= 2.0 ** -8 * diff.abs() + 1e-6 * scale).all()
    dws = (loss(g64, w64 + h) - loss(g64, w64 - h)) / (2 * h)
    assert ((dw.double() - dws).abs() <= 1e-5 * (1 + dws.abs())).all()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("P,I", [(1, 16), (1, 512), (70, 144), (33, 2048), (600, 512)])
def test_swiglu_in_8_bits(ft, P, I, weighted):
    """Scales within the fp32 error of h; every value within half an e4m3 step (2^-4 of it, or of the
    block's 2^-9 scale steps) of the formula's."""
    gu, _, w = _inputs(P, I, weighted, seed=3)
    codes = torch.empty((P, I), dtype=torch.uint8, device="cuda")
    scales = torch.empty((-(-I // 128), P), device="cuda")
    ft.ft_moe_swiglu_quantize_fp8(gu, w, codes, scales)
    h = _formula(gu, w)
    nb = scales.shape[0]
    amax = torch.nn.functional.pad(h, (0, nb * 128 - I)).view(P, nb, 128).abs().amax(2).t()
    assert ((scales.double() - amax / 448).abs() <= 2.0 ** -19 * amax / 448 + 2.0 ** -126).all()
    s = scales.double().t().repeat_interleave(128, 1)[:, :I]
    value = codes.view(torch.float8_e4m3fn).double() * s
    assert ((value - h).abs() <= (2.0 ** -4 + 2.0 ** -18) * h.abs() + 2.0 ** -10 * s * 1.001).all()


def test_extreme_gates(ft):
    """silu of large negative gates is a (negative) zero, of large positive ones the gate."""
    g = torch.tensor([-3e38, -1000.0, -90.0, -50.0, 0.0, 50.0, 1000.0, 3e38] * 2)
    gu = torch.cat([g, torch.ones(16)])[None].bfloat16().cuda()
    h = torch.empty((1, 16), dtype=torch.bfloat16, device="cuda")
    ft.ft_moe_swiglu(gu, None, h)
    ref = torch.tensor([0, 0, 0, -50 * 1.9287e-22, 0, 50, 1000, float(gu[0, 7])] * 2, dtype=torch.float64)
    assert torch.isfinite(h).all()
    assert ((h[0].double().cpu() - ref).abs() <= 0.01 * ref.abs() + 1e-30).all()
    dgu = torch.empty((1, 32), dtype=torch.bfloat16, device="cuda")
    ft.ft_moe_swiglu_backward(gu, None, torch.ones_like(h), dgu)
    assert torch.isfinite(dgu).all()
