"""Sums along a row count every column, once: rows with one value that is not zero, each in another column, where a sum is
that one term and whatever else the kernel adds or leaves out changes the result by its whole size; and sums of all columns
within the roundings that the kernels make.

Tolerances (u = 2^-24, a rounding to fp32). A sum of squares: at most 16 multiply-adds a thread, 5 + 5 additions over the
lanes and the warps, all of one sign: 26 u. The mean's division and the addition of eps: 28 u. rstd, half of that and its
own rounding: 15 u. y: three more (the gain, two products), and the store's 2^-8: 18 u + 2^-8. A scale (of 448) two more
than y's 18 u before its store.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
u = 2.0 ** -24


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


# every kernel variant and its edges; odd widths go an element at a time
WIDTHS = [1, 8, 31, 255, 256, 257, 264, 1024, 1025, 1032, 2047, 2048, 2056, 4095, 4096, 4104, 5000, 8191, 8192, 8193, 8200,
          16383, 16384]


def _diagonal(H, value, dtype):
    """[H, H] with value[c] at (c, c) and zeros elsewhere."""
    t = torch.zeros((H, H), dtype=dtype, device="cuda")
    t.diagonal().copy_(value)
    return t


def _distinct(H):
    """1, 1.125 .. 2.5: exact in bf16, neighbours differ."""
    return 1 + torch.arange(H, device="cuda") % 13 / 8


@pytest.mark.parametrize("of", ["x", "bf16 residual", "f32 residual"])
@pytest.mark.parametrize("H", WIDTHS)
def test_every_column_of_the_sum_of_squares(ft, H, of):
    v = _distinct(H)
    kind = F32 if of == "f32 residual" else BF
    x = _diagonal(H, v, BF) if of == "x" else torch.zeros((H, H), dtype=BF, device="cuda")
    r = None if of == "x" else _diagonal(H, v, kind)
    total = None if r is None else torch.empty((H, H), dtype=kind, device="cuda")
    w = torch.ones(H, device="cuda")
    y, rstd = torch.empty((H, H), dtype=BF, device="cuda"), torch.empty(H, device="cuda")
    coded = {}
    if H % 16 == 0:
        coded = dict(codes=torch.empty((H, H), dtype=U8, device="cuda"), scales=torch.empty(((H + 127) // 128, H), device="cuda"))
    for extra in ([{}, coded] if coded else [{}]):
        y.fill_(7.0)
        rstd.fill_(-1.0)
        ft.ft_moe_rmsnorm(x, w, EPS, y=y, residual=r, total=total, rstd=rstd, **extra)
        ref = (v.double().pow(2) / H + torch.tensor(EPS, dtype=F32).double().item()).rsqrt()
        assert ((rstd.double() - ref).abs() <= 15.5 * u * ref).all()
        yref = v.double() * ref
        assert ((y.diagonal().double() - yref).abs() <= (2.0 ** -8 + 19 * u) * yref).all()
        assert int(y.count_nonzero()) == H
    if coded:
        c = torch.arange(H, device="cuda")
        s = coded["scales"][c // 128, c].double()
        assert ((s - yref / 448).abs() <= 21 * u * yref / 448).all()
        # the largest value of its block: code 448 (0x7E), all others 0
        assert (coded["codes"].diagonal() == 0x7E).all() and int(coded["codes"].count_nonzero()) == H


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_sums_of_squares_of_whole_rows(ft, H, kind):
    gen = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn((50, H), generator=gen, device="cuda").bfloat16()
    r = torch.randn((50, H), generator=gen, device="cuda").to(kind)
    w = torch.randn(H, generator=gen, device="cuda")
    total, y, rstd = torch.empty_like(r), torch.empty_like(x), torch.empty(50, device="cuda")
    ft.ft_moe_rmsnorm(x, w, EPS, y=y, residual=r, total=total, rstd=rstd)
    t = total.double()
    ref = (t.pow(2).mean(1) + torch.tensor(EPS, dtype=F32).double().item()).rsqrt()
    assert ((rstd.double() - ref).abs() <= 15.5 * u * ref).all()
    yref = t * ref[:, None] * w.double()
    assert ((y.double() - yref).abs() <= (2.0 ** -8 + 19 * u) * yref.abs() + 1e-38).all()


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_every_column_of_the_norms_gradient(ft, H, kind):
    """total all ones, rstd 1, dy one value a row: mean(g n) is that value's g / H in every row (one division: u), dx is -g / H
    beside it and g - g / H at it (a multiply-add: u each, and the store), and dw[c] is row c's value, as it is."""
    v = _distinct(H)
    dy, total = _diagonal(H, v, BF), torch.ones((H, H), dtype=kind, device="cuda")
    w = 1 + torch.arange(H, device="cuda") % 7 / 8
    rstd = torch.ones(H, device="cuda")
    dx, dw = torch.empty((H, H), dtype=kind, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(ft.ft_moe_rmsnorm_workspace_size(H, H), dtype=U8, device="cuda")
    ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, dx, ws, dw=dw)
    g = v.double() * w.double()
    store = 2.0 ** -8 if kind == BF else u
    for at in range(0, H, 2048):
        rows = slice(at, min(at + 2048, H))
        got, c = dx[rows].double(), (g[rows] / H)[:, None]
        ref = (-c).repeat(1, H)
        ref.diagonal(at).add_(g[rows])
        # (c is off by u and its product with n = 1 is exact; the sum at the value itself rounds once more)
        assert ((got - ref).abs() <= store * 1.01 * ref.abs() + 2 * u * c + u * ref.abs()).all()
    assert torch.equal(dw, v)


@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_every_column_of_the_routing_weights_gradient(ft, H, dt, yt):
    """One value a row of y: dw[s] is its product with dout's, which fp32 holds (both have four bits)."""
    v, d = _distinct(H), 1 + torch.arange(H, device="cuda") % 7 / 8
    y, dout = _diagonal(H, v, yt), d.to(dt).repeat(H, 1)
    pos = torch.randperm(H, generator=torch.Generator(device="cuda").manual_seed(H), device="cuda").int().view(H, 1)
    dy, dw = torch.empty((H, H), dtype=BF, device="cuda"), torch.full((H, 1), -1.0, device="cuda")
    ft.ft_moe_combine_backward(dout, y, pos, None, dy, dw=dw)
    at = pos[:, 0].long()
    assert torch.equal(dw[:, 0], v[at] * d[at])
