"""Calls whose output is one of their inputs (total the residual, dx the gradient past the norm, out the added rows) give the
bits of calls with an output apart, over many rows, with rows that share 32-byte sectors and 128-byte lines with rows of other
CTAs, on several runs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


def _rows(gen, rows, H, lead, kind):
    """[rows, H], `lead` elements behind a 16-byte boundary, without gaps between the rows."""
    flat = torch.randn(rows * H + lead, generator=gen, device="cuda").to(kind)
    return flat[lead:].view(rows, H)


# every kernel variant (threads per row, one or two vectors a thread), whole vectors and single elements
SIZES = [(4000, 24, 0), (4000, 33, 1), (3000, 256, 0), (2000, 257, 1), (2000, 1024, 0), (2000, 1023, 1), (1500, 2048, 0),
         (1500, 2047, 1), (999, 4096, 0), (999, 4095, 3), (400, 8192, 0), (400, 8191, 1), (200, 16384, 0), (200, 16383, 1)]


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("rows,H,lead", SIZES)
def test_total_over_the_residual(ft, rows, H, lead, kind):
    gen = torch.Generator(device="cuda").manual_seed(rows + H)
    x, r = _rows(gen, rows, H, lead, BF), _rows(gen, rows, H, lead, kind)
    w = torch.randn(H, generator=gen, device="cuda")
    total, y, rstd = torch.empty((rows, H), dtype=kind, device="cuda"), torch.empty_like(x), torch.empty(rows, device="cuda")
    ft.ft_moe_rmsnorm(x, w, EPS, y=y, residual=r, total=total, rstd=rstd)
    y2, rstd2 = torch.empty_like(y), torch.empty_like(rstd)
    for _ in range(3):
        both = _rows(gen, rows, H, lead, kind)
        both.copy_(r)
        ft.ft_moe_rmsnorm(x, w, EPS, y=y2, residual=both, total=both, rstd=rstd2)
        assert torch.equal(both, total) and torch.equal(y2, y) and torch.equal(rstd2, rstd)


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("rows,H,lead", SIZES)
def test_dx_over_the_gradient_past_the_norm(ft, rows, H, lead, kind):
    gen = torch.Generator(device="cuda").manual_seed(rows + 2 * H)
    total, dy, past = _rows(gen, rows, H, lead, kind), _rows(gen, rows, H, lead, BF), _rows(gen, rows, H, lead, kind)
    w, rstd = torch.randn(H, generator=gen, device="cuda"), torch.rand(rows, generator=gen, device="cuda") + 0.5
    dx = torch.empty((rows, H), dtype=kind, device="cuda")
    ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, dx, dtotal=past)
    for _ in range(3):
        both = _rows(gen, rows, H, lead, kind)
        both.copy_(past)
        ft.ft_moe_rmsnorm_backward(dy, total, w, rstd, both, dtotal=both)
        assert torch.equal(both, dx)


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("rows,H,lead", SIZES)
def test_out_over_the_added_rows(ft, rows, H, lead, kind):
    gen, k = torch.Generator(device="cuda").manual_seed(rows + 3 * H), 3
    y, add = _rows(gen, rows * k, H, lead, BF), _rows(gen, rows, H, lead, kind)
    pos = torch.randperm(rows * k, generator=gen, device="cuda").int().view(rows, k)
    w = torch.rand((rows, k), generator=gen, device="cuda")
    out = torch.empty((rows, H), dtype=kind, device="cuda")
    ft.ft_moe_combine(y, pos, w, out, add=add)
    for _ in range(3):
        both = _rows(gen, rows, H, lead, kind)
        both.copy_(add)
        ft.ft_moe_combine(y, pos, w, both, add=both)
        assert torch.equal(both, out)
