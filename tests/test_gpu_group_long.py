"""Weight gradients of very long contractions (millions of rows of one expert), stored in bf16:
the sums are fp32 sums however many rows there are.

All products are positive, so that what an addition loses adds up. An fp32 sum of 4096 steps in
the tensor cores loses at most 256 times 2^-23 of itself (one truncation per instruction of 16
steps), the sum of up to 1024 such parts (and of a cluster's eight) at most 2^-24 each:
2^-15 + 2^-14 + 2^-21, and the store half an ulp of bf16.
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


# one expert whose rows a cluster shares; one of many, its rows a pair's or a single thread block's
@pytest.mark.parametrize("E,P,N,K", [(1, 1 << 24, 64, 64), (40, 1 << 22, 256, 256), (40, 1 << 22, 256, 128)])
def test_bf16_wgrad_of_millions_of_rows(ft, E, P, N, K):
    gen = torch.Generator(device="cuda").manual_seed(E)
    e = E // 2
    # factors from 1 to 2 spread the sums over a binade: every distance to a rounding boundary occurs
    x = torch.rand((P, K), generator=gen, device="cuda", dtype=torch.bfloat16) * torch.linspace(1, 2, K, device="cuda").bfloat16()
    dy = torch.rand((P, N), generator=gen, device="cuda", dtype=torch.bfloat16)
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[e + 1:] = P
    dw = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device="cuda")
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws)
    assert ft.ft_moe_read_status(ws) == 0
    ref = torch.zeros((N, K), dtype=torch.float64, device="cuda")
    for a, b in zip(dy.split(1 << 18), x.split(1 << 18)):
        ref += a.double().t() @ b.double()
    half_ulp = torch.exp2(torch.floor(torch.log2(ref)) - 8)
    err = (dw[e].double() - ref).abs()
    assert (err <= half_ulp + (2.0 ** -14 + 2.0 ** -15 + 2.0 ** -21) * ref).all(), float((err / ref).max())
    dw[e] = 0
    assert not dw.any()


@pytest.mark.parametrize("N,K", [(136, 72), (200, 264), (264, 520)])
def test_bf16_wgrad_of_many_rows_of_ragged_experts(ft, N, K):
    """More than 65536 rows, over experts with none to thousands: products are exact in fp32, a sum of R is
    within R * 2^-23 of the magnitudes, the store rounds to 2^-8. Experts with rows that are not finite
    keep them to themselves; repeats are equal to the bit."""
    sizes = [(37 * i) % 700 for i in range(200)] + [0, 9000, 1, 4097]
    gen = torch.Generator(device="cuda").manual_seed(3)
    P, E = sum(sizes), len(sizes)
    assert P > 65536
    x, dy = (torch.randn((P, c), generator=gen, device="cuda").bfloat16() for c in (K, N))
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    bad = [30, 100, 202]
    for e in bad:
        x[at[e]:at[e + 1]], dy[at[e]:at[e + 1]] = float("nan"), float("inf")
    offs = torch.tensor(at, dtype=torch.int32, device="cuda")
    ws = torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device="cuda")
    dw, again = (torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, dw, ws)
    assert ft.ft_moe_read_status(ws) == 0
    ft.ft_moe_group_gemm_wgrad(dy, x, offs, again, ws)
    assert torch.equal(dw.view(torch.int16), again.view(torch.int16))
    for e, n in enumerate(sizes):
        if e in bad:
            assert not torch.isfinite(dw[e]).any()
            continue
        a, b = dy[at[e]:at[e + 1]].double(), x[at[e]:at[e + 1]].double()
        ref, mag = a.t() @ b, a.abs().t() @ b.abs()
        assert ((dw[e].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + n * 2.0 ** -23 * mag).all(), e
