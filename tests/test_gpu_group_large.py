"""The expert products at the ends of their ranges: 1024 experts, and operands and outputs of more than
2^31 elements in every direction and type. Tolerances as in the arithmetic: R * 2^-23 of the
magnitudes for a sum of R products (8-bit products four more), and one rounding at the store."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ft():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    yield ft
    torch.cuda.empty_cache()


def _ws(ft, E, P, N, K):
    return torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device="cuda")


def _near(got, a, b, R, extra=0.0):
    """got = a . b, summed over R."""
    ref, mag = a @ b, a.abs() @ b.abs()
    if torch.is_tensor(extra):
        ref, mag, R = ref + extra, mag + extra.abs(), R + 1
    assert ((got.double() - ref).abs() <= U[got.dtype] * ref.abs() + R * 2.0 ** -23 * mag + 1e-30).all()


@pytest.mark.parametrize("most", [3, 60, 400])
def test_1024_experts(ft, most):
    """One row for a third of them, none for a third, up to `most` for the others."""
    E, N, K = 1024, 136, 272
    sizes = [(0, 1, (31 * i) % (most + 1))[i % 3] for i in range(E)]
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    P = at[-1]
    gen = torch.Generator(device="cuda").manual_seed(most)
    x, dy, w = (torch.randn(s, generator=gen, device="cuda").bfloat16() for s in ((P, K), (P, N), (E, N, K)))
    offs, ws = torch.tensor(at, dtype=torch.int32, device="cuda"), _ws(ft, E, P, N, K)
    y, dx = torch.empty((P, N), device="cuda"), torch.empty((P, K), dtype=BF, device="cuda")
    dw, base = torch.empty((E, N, K), dtype=BF, device="cuda"), torch.randn((E, N, K), generator=gen, device="cuda")
    added, y8 = base.clone(), torch.empty((P, N), dtype=BF, device="cuda")
    q, qs = torch.empty((P, K), dtype=torch.uint8, device="cuda"), torch.empty((3, P), device="cuda")
    wq, wsc = w.float().to(torch.float8_e4m3fn), torch.rand((E, 2, 3), generator=gen, device="cuda") + 0.1
    for call in (lambda: ft.ft_moe_group_gemm(x, w, offs, y, ws), lambda: ft.ft_moe_group_gemm_dgrad(dy, w, offs, dx, ws),
                 lambda: ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws),
                 lambda: ft.ft_moe_group_gemm_wgrad(dy, x, offs, added, ws, accumulate=True),
                 lambda: ft.ft_moe_quantize_fp8(x, q, qs),
                 lambda: ft.ft_moe_group_gemm_fp8(q, qs, wq, wsc, offs, y8, ws)):
        call()
        assert ft.ft_moe_read_status(ws) == 0
    xd = q.view(torch.float8_e4m3fn).double() * qs.double().t().repeat_interleave(128, 1)[:, :K]
    for e in list(range(0, E, 37)) + [1, 2, E - 2, E - 1]:
        r = slice(at[e], at[e + 1])
        xe, de, we = x[r].double(), dy[r].double(), w[e].double()
        _near(y[r], xe, we.t(), K)
        _near(dx[r], de, we, N)
        _near(dw[e], de.t(), xe, sizes[e])
        _near(added[e], de.t(), xe, sizes[e], base[e].double())
        scale = wsc[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        _near(y8[r], xd[r], (wq[e].double() * scale).t(), K + 4)


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", ["forward", "dgrad", "8-bit"])
def test_rows_beyond_2_to_31(ft, form, out):
    P, wide, R = 1 << 18, 8448, 64   # 2.2e9 outputs
    N, K = (R, wide) if form == "dgrad" else (wide, R)
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, w = (torch.randn(s, generator=gen, device="cuda").bfloat16() for s in ((P, R), (2, N, K)))
    offs = torch.tensor([0, P - 300, P], dtype=torch.int32, device="cuda")
    y, ws = torch.empty((P, wide), dtype=out, device="cuda"), _ws(ft, 2, P, N, K)
    rows = torch.cat([torch.arange(200), torch.arange(P - 500, P)]).cuda()
    left, right = a[rows].double(), w.double()
    if form == "forward":
        ft.ft_moe_group_gemm(a, w, offs, y, ws)
        right = right.transpose(1, 2)
    elif form == "dgrad":
        ft.ft_moe_group_gemm_dgrad(a, w, offs, y, ws)
    else:
        q, qs = torch.empty((P, R), dtype=torch.uint8, device="cuda"), torch.empty((1, P), device="cuda")
        ft.ft_moe_quantize_fp8(a, q, qs)
        wq = w.float().to(torch.float8_e4m3fn)
        ft.ft_moe_group_gemm_fp8(q, qs, wq, torch.ones((2, N // 128, 1), device="cuda"), offs, y, ws)
        left = q[rows].view(torch.float8_e4m3fn).double() * qs[0, rows, None].double()
        right = wq.double().transpose(1, 2)
    assert ft.ft_moe_read_status(ws) == 0
    got = y[rows]
    _near(got[:400], left[:400], right[0], R + 4)
    _near(got[400:], left[400:], right[1], R + 4)


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradients_beyond_2_to_31(ft, accumulate):
    E, N, K = 520, 2048, 2048
    gen = torch.Generator(device="cuda").manual_seed(2)
    sizes = [200] + [0] * (E - 3) + [300, 25]
    P = sum(sizes)
    x, dy = (torch.randn((P, c), generator=gen, device="cuda").bfloat16() for c in (K, N))
    offs = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    dw, ws = torch.full((E, N, K), 2.0, device="cuda"), _ws(ft, E, P, N, K)
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws, accumulate=accumulate)
    assert ft.ft_moe_read_status(ws) == 0
    start = torch.full((N, K), 2.0 if accumulate else 0.0, dtype=torch.float64, device="cuda")
    for e, rows in ((0, slice(0, 200)), (E - 2, slice(200, 500)), (E - 1, slice(500, 525))):
        _near(dw[e], dy[rows].double().t(), x[rows].double(), rows.stop - rows.start, start)
    for part in dw[1:E - 2].split(40):
        assert (part == (2.0 if accumulate else 0.0)).all()
