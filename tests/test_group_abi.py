"""Argument checks of the expert products and row kernels: everything a call can refuse is refused
on the host, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

A = 4096  # an aligned stand-in address; nothing is launched in these tests


@pytest.fixture(scope="module")
def ft():
    from nvfp4_quantized_moe_gb300 import build
    build.build()
    import nvfp4_quantized_moe_gb300 as ft
    ft.load()
    return ft


FORWARD = dict(x=A, ld_x=64, w=A, offs=A, E=2, P=8, N=128, K=64, y=A, ld_y=128, dtype=3, ws=A, ws_bytes=256, stream=None)
DGRAD = dict(dy=A, ld_dy=128, w=A, offs=A, E=2, P=8, N=128, K=64, dx=A, ld_dx=64, dtype=3, ws=A, ws_bytes=256, stream=None)
WGRAD = dict(dy=A, ld_dy=128, x=A, ld_x=64, offs=A, E=2, P=8, N=128, K=64, dw=A, dtype=2, accumulate=0, ws=A, ws_bytes=256,
             stream=None)
FP8 = dict(x=A, ld_x=64, xs=A, ld_xs=8, w=A, wscale=A, offs=A, E=2, P=8, N=128, K=64, y=A, ld_y=128, dtype=3, ws=A,
           ws_bytes=256, stream=None)
QUANT = dict(src=A, dtype=3, ld=64, rows=4, K=64, codes=A, ld_codes=64, scales=A, ld_scales=4, stream=None)
SWIGLU = dict(gu=A, ld_gu=128, w=A, rows=4, I=64, h=A, ld_h=64, stream=None)
SWIGLU8 = dict(gu=A, ld_gu=128, w=A, rows=4, I=64, codes=A, ld_codes=64, scales=A, ld_scales=4, stream=None)
BACKWARD = dict(gu=A, ld_gu=128, w=A, dh=A, ld_dh=64, rows=4, I=64, dgu=A, ld_dgu=128, dw=A, stream=None)

CALLS = {"ft_moe_group_gemm": FORWARD, "ft_moe_group_gemm_dgrad": DGRAD, "ft_moe_group_gemm_wgrad": WGRAD,
         "ft_moe_group_gemm_fp8": FP8, "ft_moe_quantize_fp8": QUANT, "ft_moe_swiglu": SWIGLU,
         "ft_moe_swiglu_quantize_fp8": SWIGLU8, "ft_moe_swiglu_backward": BACKWARD}

GROUP = [(dict(E=0), 1), (dict(E=1025), 3), (dict(P=-1), 1), (dict(P=(1 << 25) + 1), 3), (dict(N=0), 1), (dict(K=-8), 1),
         (dict(N=65544), 3), (dict(K=65552), 3), (dict(offs=None), 1), (dict(offs=A + 2), 1), (dict(dtype=0), 1),
         (dict(ws=None), 1), (dict(ws=A + 16), 1), (dict(ws_bytes=255), 4)]
CASES = (
    [("ft_moe_group_gemm", *c) for c in GROUP + [(dict(N=12), 3), (dict(K=20), 3), (dict(x=None), 1), (dict(x=A + 8), 1),
                                                 (dict(w=A + 2), 1), (dict(y=None), 1), (dict(ld_x=56), 1), (dict(ld_x=68), 1),
                                                 (dict(ld_y=120), 1), (dict(ld_y=132), 1)]]
    + [("ft_moe_group_gemm_dgrad", *c) for c in GROUP + [(dict(dy=None), 1), (dict(ld_dy=64), 1), (dict(dx=A + 4), 1),
                                                         (dict(ld_dx=60), 1), (dict(w=None), 1)]]
    + [("ft_moe_group_gemm_wgrad", *c) for c in GROUP + [(dict(accumulate=2), 1), (dict(accumulate=1, dtype=3), 3),
                                                         (dict(dw=None), 1), (dict(dy=A + 8), 1), (dict(ld_x=32), 1)]]
    + [("ft_moe_group_gemm_fp8", *c) for c in GROUP + [(dict(K=72, ld_x=80), 3), (dict(ld_x=72), 1), (dict(xs=None), 1),
                                                       (dict(wscale=A + 2), 1), (dict(ld_xs=7), 1), (dict(ld_y=127), 1),
                                                       (dict(w=A + 8), 1)]]
    + [("ft_moe_quantize_fp8", *c) for c in [(dict(dtype=0), 1), (dict(rows=-1), 1), (dict(K=0), 1), (dict(K=72), 3),
                                             (dict(src=None), 1), (dict(src=A + 8), 1), (dict(ld=60), 1), (dict(codes=A + 8), 1),
                                             (dict(ld_codes=72), 1), (dict(scales=None), 1), (dict(ld_scales=3), 1)]]
    + [("ft_moe_swiglu", *c) for c in [(dict(rows=-1), 1), (dict(I=0), 1), (dict(I=70000), 3), (dict(gu=None), 1),
                                       (dict(gu=A + 1), 1), (dict(ld_gu=127), 1), (dict(h=None), 1), (dict(ld_h=63), 1),
                                       (dict(w=A + 2), 1)]]
    + [("ft_moe_swiglu_quantize_fp8", *c) for c in [(dict(I=72), 3), (dict(gu=A + 2), 1), (dict(ld_gu=132), 1),
                                                    (dict(codes=None), 1), (dict(scales=A + 2), 1), (dict(w=A + 1), 1)]]
    + [("ft_moe_swiglu_backward", *c) for c in [(dict(dh=None), 1), (dict(ld_dh=63), 1), (dict(dgu=A + 1), 1),
                                                (dict(ld_dgu=100), 1), (dict(dw=A + 2), 1), (dict(I=-1), 1)]]
)


@pytest.mark.parametrize("name,change,code", CASES, ids=[f"{n[7:]}-{c}" for n, c, _ in CASES])
def test_refusals(ft, name, change, code):
    args = dict(CALLS[name], **change)
    assert getattr(ft.load(), name)(*args.values()) == code
    assert ft.ft_last_error()


@pytest.mark.parametrize("name,change", [("ft_moe_quantize_fp8", dict(src=None, codes=None, scales=None)),
                                         ("ft_moe_swiglu", dict(gu=None, h=None)),
                                         ("ft_moe_swiglu_quantize_fp8", dict(gu=None, codes=None, scales=None)),
                                         ("ft_moe_swiglu_backward", dict(gu=None, dh=None, dgu=None))])
def test_no_rows_is_a_no_op(ft, name, change):
    assert getattr(ft.load(), name)(*dict(CALLS[name], rows=0, **change).values()) == 0
    assert ft.ft_last_error() == ""


def test_workspace_size(ft):
    n = ctypes.c_size_t()
    assert ft.ft_moe_group_workspace_size(256, 512, 1024, 2048) >= 256
    assert ft.load().ft_moe_group_workspace_size(256, 512, 1024, 2048, None) == 1
    assert ft.load().ft_moe_group_workspace_size(0, 512, 1024, 2048, ctypes.byref(n)) == 1
    assert ft.load().ft_moe_group_workspace_size(2048, 512, 1024, 2048, ctypes.byref(n)) == 3


def test_binding_refuses_what_it_cannot_pass(ft):
    """Types, shapes and layouts the C call cannot see."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ws, offs = torch.zeros(256, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    x, w, y = bf(8, 64), bf(2, 128, 64), bf(8, 128)
    bad = [
        lambda: ft.ft_moe_group_gemm(x.float(), w, offs, y, ws),
        lambda: ft.ft_moe_group_gemm(x[:, :32], w, offs, y, ws),
        lambda: ft.ft_moe_group_gemm(bf(64, 8).t(), w, offs, y, ws),
        lambda: ft.ft_moe_group_gemm(x, w.transpose(1, 2), offs, bf(8, 64), ws),
        lambda: ft.ft_moe_group_gemm(x, w, offs, y[:4], ws),
        lambda: ft.ft_moe_group_gemm(x, w, offs.long(), y, ws),
        lambda: ft.ft_moe_group_gemm(x, w, offs[:2], y, ws),
        lambda: ft.ft_moe_group_gemm(x, w, None, y, ws),
        lambda: ft.ft_moe_group_gemm(x, w, offs, y.half(), ws),
        lambda: ft.ft_moe_group_gemm_wgrad(y, x[:4], offs, w, ws),
        lambda: ft.ft_moe_group_gemm_fp8(x.byte(), torch.zeros(8, 1), w.byte(), torch.zeros(2, 1, 1), offs, y, ws),
        lambda: ft.ft_moe_group_gemm_fp8(x.byte(), torch.zeros(1, 8), w.byte(), torch.zeros(2, 1, 2), offs, y, ws),
        lambda: ft.ft_moe_quantize_fp8(x, x.byte()[:, :32], torch.zeros(1, 8)),
        lambda: ft.ft_moe_swiglu(y, torch.zeros(7), x),
        lambda: ft.ft_moe_swiglu(y, torch.zeros(8, dtype=torch.float64), x),
        lambda: ft.ft_moe_swiglu_backward(y, None, x, bf(8, 64)),
        lambda: ft.ft_moe_group_gemm(x, w, offs, y, ws),   # all well formed, but not on the GPU
        lambda: ft.ft_moe_swiglu(y, None, x),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_plan_refusals(ft):
    plan = (ctypes.c_int32 * 4)()
    call = ft.load().ft_moe_debug_group_plan
    good = dict(product=2, E=2, P=8, N=128, K=64, dtype=2, accumulate=1, plan=plan)
    for change, code in ((dict(product=-1), 1), (dict(product=4), 1), (dict(P=0), 1), (dict(plan=None), 1), (dict(accumulate=2), 1),
                         (dict(dtype=3), 1), (dict(product=0), 1), (dict(dtype=0, accumulate=0), 1), (dict(E=0), 1),
                         (dict(N=12), 3), (dict(product=3, accumulate=0, K=72), 3), (dict(E=1025), 3)):
        assert call(*dict(good, **change).values()) == code, change
        assert ft.ft_last_error()
