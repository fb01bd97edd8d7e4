"""MXFP4: quantizers, scale tiles and the grouped product, through the C ABI.

Quantizers are compared bit for bit with the rule (exact scaling, so that there is nothing to be off by). In the product
every term is exact; the tensor cores add 64 of them and an fp32 accumulator per instruction, truncating to a few bits
beyond fp32's: (K / 64 + 8) additions, each off by at most 2^-22 of the terms' magnitudes, and the store's 2^-8 (bf16) or
2^-24 of the result.
"""
import pytest
import torch

from mxfp4_cases import codes_of, decode, random_weights, row_scales, rule, tiles_of, words_of

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantize(ft, x):
    codes, scales = torch.empty((x.shape[0], x.shape[1] // 2), dtype=U8, device="cuda"), ft.alloc_mxfp4_scales(*x.shape)
    ft.ft_moe_quantize_mxfp4(x, codes, scales)
    return codes, scales


def _same_codes(a, b):
    return ((a == b) | ((a & 7 == 0) & (b & 7 == 0))).all()  # (zero of either sign)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,K,pad", [(1, 32, 0), (1, 2048, 0), (3, 128, 0), (17, 160, 8), (100, 2016, 0), (33, 4096, 16), (5000, 96, 0)])
def test_quantizer_is_bit_exact(ft, P, K, pad, dtype):
    gen = _gen(P + K)
    x = torch.randn((P, K + pad), generator=gen, device="cuda")
    x = x * torch.exp2(torch.randint(-40, 40, (P, 1), generator=gen, device="cuda").float())
    x = x.to(dtype)
    if P > 2:
        x[1], x[2, :32] = 0, 0
        x[0, :15] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0])
        x[0, 15:32] = 0
    codes = torch.full((P, K // 2 + 16), 0xAA, dtype=U8, device="cuda")
    scales = torch.full(((K + 127) // 128, (P + 7) // 4 * 4, 4), 0xBB, dtype=U8, device="cuda")
    ft.ft_moe_quantize_mxfp4(x[:, :K], codes[:, :K // 2], scales[:, :P])
    ref_c, ref_s = rule(x[:, :K].float())
    assert torch.equal(row_scales(scales[:, :P], K), ref_s)
    assert torch.equal(scales[:, :P], words_of(ref_s))  # (zeros beyond K)
    assert _same_codes(codes_of(codes[:, :K // 2]).int(), ref_c)
    assert (codes[:, K // 2:] == 0xAA).all() and (scales[:, P:] == 0xBB).all()


def test_quantizer_edges(ft):
    """Every border of the scale rule, the limits of fp32, and values that are not finite (their block alone)."""
    x = torch.zeros((8, 64))
    x[0, 0], x[0, 32] = 1.5, 1.5 + 2.0 ** -20
    x[1, 0], x[1, 32] = 2.0 ** -126, 2.0 ** -140
    x[2, 0], x[2, 32] = 3.4e38, -2.0 ** 127
    x[3, 3], x[3, 40] = float("inf"), 1.0
    x[4, 3], x[4, 40] = 1.0, float("nan")
    x[5, 0], x[5, 32] = 6.0 * 2.0 ** -127, 6.1 * 2.0 ** -127
    x[6, 0], x[6, 32] = -0.0, 1e-45
    x[7, :] = torch.linspace(-6, 6, 64)
    x = x.cuda()
    codes, scales = _quantize(ft, x)
    ref_c, ref_s = rule(x)
    assert torch.equal(row_scales(scales, 64), ref_s)
    assert ref_s[3, 0] == 255 and ref_s[4, 1] == 255 and ref_s[3, 1] != 255 and ref_s[4, 0] != 255
    fine = (ref_s != 255).repeat_interleave(32, 1)
    assert _same_codes(codes_of(codes).int()[fine], ref_c[fine])
    value = decode(codes, row_scales(scales, 64))
    assert torch.isnan(value[~fine]).all()
    amax = x.double().view(8, 2, 32).abs().amax(2).repeat_interleave(32, 1)
    assert ((value - x.double()).abs()[fine] <= 0.25 * x.double().abs()[fine] + (amax / 24 + 2.0 ** -129)[fine]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (3, 200, 96), (2, 5, 2048), (4, 640, 544)])
def test_weight_quantizer_and_packing(ft, E, N, K, dtype):
    """Weights come out as their rows would, with the scales in tiles; packing row-major scales gives the same tiles."""
    w = (torch.randn((E, N, K), generator=_gen(N), device="cuda") * 0.02).to(dtype)
    codes = torch.empty((E, N, K // 2), dtype=U8, device="cuda")
    tiles = torch.zeros((E, (N + 127) // 128, (K + 127) // 128, 512), dtype=U8, device="cuda")
    ft.ft_moe_quantize_mxfp4_weights(w, codes, tiles)
    rc, rs = _quantize(ft, w.view(E * N, K))
    scales = row_scales(rs, K).contiguous().view(E, N, K // 32)
    assert torch.equal(codes, rc.view(E, N, K // 2)) and torch.equal(tiles, tiles_of(scales))
    packed = torch.full_like(tiles, 0xCC)
    ft.ft_moe_pack_mxfp4_scales(scales, packed)
    assert torch.equal(packed, tiles)
    ft.ft_moe_pack_mxfp4_scales(scales.view(torch.float8_e8m0fnu), packed)
    assert torch.equal(packed, tiles)


def _silu(gu, w):
    g, u = gu.double().chunk(2, 1)
    return (1.0 if w is None else w.double()[:, None]) * g * torch.sigmoid(g) * u


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("P,I", [(1, 32), (1, 512), (70, 160), (33, 2048), (600, 512)])
def test_swiglu(ft, P, I, weighted):
    """Scales are powers of two that hold the block and whose halves do not, within the fp32 error of h (2^-19); values
    are off by half a step: a quarter of the value, or a quarter of the scale near zero."""
    gen = _gen(P + I)
    gu = (torch.randn((P, 2 * I), generator=gen, device="cuda") * 2).bfloat16()
    w = torch.rand(P, generator=gen, device="cuda") if weighted else None
    codes, scales = torch.empty((P, I // 2), dtype=U8, device="cuda"), ft.alloc_mxfp4_scales(P, I)
    ft.ft_moe_swiglu_quantize_mxfp4(gu, w, codes, scales)
    h = _silu(gu, w)
    byte = row_scales(scales, I)
    s = torch.exp2(byte.double() - 127)
    amax, eps = h.view(P, -1, 32).abs().amax(2), 2.0 ** -19
    assert (amax <= 6 * s * (1 + eps)).all() and ((amax >= 3 * s * (1 - eps)) | (byte == 0)).all()
    value, s = decode(codes, byte), s.repeat_interleave(32, 1)
    assert ((value - h).abs() <= (0.25 + eps) * h.abs() + 0.25 * 1.001 * s).all()
    step = torch.where(h.abs() >= 4 * s * (1 - eps), 2.0, torch.where(h.abs() >= 2 * s * (1 - eps), 1.0, 0.5)) * s
    assert ((value - h).abs() <= 0.5 * step + eps * h.abs()).all()


def _offsets(sizes):
    return torch.tensor([0, *sizes], device="cuda").cumsum(0).int()


def _product(ft, x, xs, w, ws, sizes, dtype, P=None, pad=0):
    """y of the grouped product, in rows pad elements longer, with its status."""
    E, N, half = w.shape
    P = x.shape[0]
    y = torch.full((P, N + pad), 7.0, dtype=dtype, device="cuda")
    work = torch.full((ft.ft_moe_group_workspace_size(E, max(P, 1), N, 2 * half),), 0xFF, dtype=U8, device="cuda")
    offs = None if sizes is None else _offsets(sizes)
    ft.ft_moe_group_gemm_mxfp4(x, xs, w, tiles_of(ws), offs, y[:, :N], work)
    assert ft.ft_moe_read_status(work) == 0
    if pad:
        assert (y[:, N:] == 7).all()
    return y[:, :N]


def _check(y, x64, w64, sizes, K):
    at = 0
    for e, n in enumerate(sizes):
        rows = x64[at:at + n]
        ref, mag = rows @ w64[e].t(), rows.abs() @ w64[e].abs().t()
        store = 2.0 ** -8 if y.dtype == BF else 2.0 ** -24
        err = (y[at:at + n].double() - ref).abs()
        assert (err <= store * 1.01 * ref.abs() + (K / 64 + 8) * 2.0 ** -22 * mag).all(), (e, float((err / mag).max()))
        at += n
    assert (y[at:] == 7).all()  # rows of no expert


# rows per expert: none, one, odd; every tile size and split; N and K with remainders
GROUPS = [
    ([1], 128, 32), ([1], 128, 256), ([3], 130, 96), ([1], 2048, 2048), ([8], 1024, 4096), ([31, 0, 2], 200, 544),
    ([0, 5, 0, 1, 17, 0], 257, 320), ([16, 24, 33], 640, 512), ([100, 0, 3, 250], 384, 672), ([129], 96, 1024),
    ([300], 256, 2048), ([1, 700, 64], 1000, 288), ([513, 511], 512, 512), ([2000, 100], 776, 256), ([1] * 40, 256, 544),
    ([33, 70, 0, 129, 51] * 8, 300, 288), ([31, 64, 65] * 12, 257, 544), ([128, 127, 1] * 20, 136, 64),
    # by pairs of CTAs: first rows at every remainder of four, tiles that end one before, at and behind their last row
    ([301, 0, 258, 3, 1023, 130], 3100, 544), ([255, 257, 256, 1, 511], 3700, 96), ([1500, 1340], 3000, 2112), ([17000], 520, 288),
    ([145] * 64, 264, 320), ([253, 254, 255, 256, 257, 258, 259], 2752, 128), ([60000, 1], 192, 64),
    # fewer weight rows than a piece of 16 bytes of y
    ([3], 1, 32), ([300, 5], 7, 96), ([50000], 1, 32), ([25000, 25003], 7, 64),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,N,K", GROUPS, ids=[f"{sum(s)}x{n}x{k}e{len(s)}" for s, n, k in GROUPS])
def test_product(ft, sizes, N, K, dtype):
    gen = _gen(N + K)
    P, E = sum(sizes), len(sizes)
    x = torch.randn((P + 3, K), generator=gen, device="cuda")  # three rows of no expert
    codes, xs = _quantize(ft, x)
    w, ws = random_weights(gen, E, N, K, 3)
    x64, w64 = decode(codes, row_scales(xs, K)), decode(w, ws)
    y = _product(ft, codes, xs, w, ws, sizes, dtype, pad=N % 5)
    _check(y, x64, w64, sizes, K)
    again = _product(ft, codes, xs, w, ws, sizes, dtype)
    assert torch.equal(again, y)
    if E == 1:
        plain = _product(ft, codes[:P], xs[:, :P], w, ws, None, dtype)
        assert torch.equal(plain, y[:P])


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 256, 288, 320])
def test_every_block_has_its_own_scale(ft, K):
    """One code and one scale differ from block to block: every block and row finds its own, by the exact sums."""
    P, N = 150, 140
    w = torch.full((1, N, K // 2), 0x22, dtype=U8, device="cuda")     # all ones
    x = torch.full((P, K // 2), 0x22, dtype=U8, device="cuda")
    gen = _gen(K)
    ws = torch.randint(124, 131, (1, N, K // 32), generator=gen, device="cuda", dtype=U8)
    xs = torch.randint(124, 131, (P, K // 32), generator=gen, device="cuda", dtype=U8)
    words = ft.alloc_mxfp4_scales(P, K)
    words.copy_(words_of(xs))
    y = _product(ft, x, words, w, ws, None, F32)
    ref = torch.exp2(xs.double() - 127) @ torch.exp2(ws[0].double() - 127).t() * 32
    assert torch.equal(y.double(), ref)


def test_values_that_are_not_finite_stay_in_their_rows(ft):
    for sizes, N, K in (([5, 20, 3], 200, 160), ([200, 140], 256, 512), ([700, 600], 300, 288)):
        gen = _gen(N)
        P, E = sum(sizes), len(sizes)
        x = torch.randn((P, K), generator=gen, device="cuda")
        clean, cs = _quantize(ft, x)
        w, ws = random_weights(gen, E, N, K)
        want = _product(ft, clean, cs, w, ws, sizes, F32)
        x[1, K - 1], x[sizes[0], 3] = float("nan"), float("inf")
        codes, xs = _quantize(ft, x)
        ws[0, 7, 0] = 255
        y = _product(ft, codes, xs, w, ws, sizes, F32)
        bad = torch.zeros((P, N), dtype=torch.bool, device="cuda")
        bad[1], bad[sizes[0]], bad[:sizes[0], 7] = True, True, True
        assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], want[~bad])


def test_extreme_scales(ft):
    """Scales far apart: products beyond fp32 are infinite, far below it zero, others exact."""
    P, N, K = 40, 128, 64
    w = torch.full((1, N, K // 2), 0x22, dtype=U8, device="cuda")
    x = torch.full((P, K // 2), 0x22, dtype=U8, device="cuda")
    ws = torch.full((1, N, 2), 127, dtype=U8, device="cuda")
    xs = torch.full((P, 2), 127, dtype=U8, device="cuda")
    ws[0, 1], xs[1] = 230, 240                      # 2^103, 2^113
    ws[0, 2], xs[2] = 60, 40                        # 2^-67, 2^-87
    words = ft.alloc_mxfp4_scales(P, K)
    words.copy_(words_of(xs))
    y = _product(ft, x, words, w, ws, None, F32)
    assert torch.isinf(y[1, 1]) and abs(float(y[2, 2])) <= 2.0 ** -126
    assert y[0, 0] == 64 and y[1, 0] == 2.0 ** 119 and y[0, 1] == 2.0 ** 109 and y[2, 0] == 2.0 ** -81 and y[0, 2] == 2.0 ** -61
    assert y[1, 2] == 2.0 ** 52 and y[2, 1] == 2.0 ** 22


def test_bad_offsets_are_reported(ft):
    gen = _gen(0)
    w, ws = random_weights(gen, 2, 128, 64)
    codes, xs = _quantize(ft, torch.randn((16, 64), generator=gen, device="cuda"))
    y, work = torch.empty((16, 128), dtype=BF, device="cuda"), torch.zeros(256, dtype=U8, device="cuda")
    for offs in ([0, 9, 5], [0, 5, 17], [-1, 5, 16]):
        ft.ft_moe_group_gemm_mxfp4(codes, xs, w, tiles_of(ws), torch.tensor(offs, dtype=torch.int32, device="cuda"), y, work)
        assert ft.STATUS[ft.ft_moe_read_status(work)] == "FT_ERR_INVALID_ROUTING"
    ft.ft_moe_group_gemm_mxfp4(codes, xs, w, tiles_of(ws), _offsets([9, 7]), y, work)
    assert ft.ft_moe_read_status(work) == 0


def test_no_rows(ft):
    w, ws = random_weights(_gen(0), 2, 128, 64)
    work = torch.full((256,), 0xFF, dtype=U8, device="cuda")
    codes, xs = torch.empty((0, 32), dtype=U8, device="cuda"), ft.alloc_mxfp4_scales(0, 64)
    ft.ft_moe_quantize_mxfp4(torch.empty((0, 64), device="cuda"), codes, xs)
    ft.ft_moe_group_gemm_mxfp4(codes, xs, w, tiles_of(ws), _offsets([0, 0]), torch.empty((0, 128), dtype=BF, device="cuda"), work)
    assert ft.ft_moe_read_status(work) == 0
