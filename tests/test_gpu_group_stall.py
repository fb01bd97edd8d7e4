"""Fault injection into the expert products stays armed until a call launches kernels."""
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


def test_refused_and_empty_calls_leave_it_armed(ft):
    N, K = 64, 128
    x, w = torch.ones((4, K), dtype=torch.bfloat16, device="cuda"), torch.ones((1, N, K), dtype=torch.bfloat16, device="cuda")
    y, ws = torch.empty((4, N), device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    ft.ft_moe_debug_inject_stall(5_000_000, 1)
    with pytest.raises(ft.FtMoeError):
        ft.ft_moe_group_gemm(x, w[:, :12].contiguous(), None, y[:, :12], ws)  # 12 columns: refused
    ft.ft_moe_group_gemm(x[:0], w, None, y[:0], ws)                           # no rows: nothing is launched
    ft.ft_moe_group_gemm(x, w, None, y, ws)
    assert ft.STATUS[ft.ft_moe_read_status(ws)] == "FT_ERR_TIMEOUT"
    ft.ft_moe_group_gemm(x, w, None, y, ws)
    assert ft.ft_moe_read_status(ws) == 0 and (y == K).all()
