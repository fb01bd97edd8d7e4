"""Argument checks of the residual norm, of the tokens' sorting and of the MXFP4 calls: everything a call can refuse is
refused on the host, before any launch (no GPU needed)."""
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


NORM = dict(x=A, ld_x=64, residual=A, ld_r=64, total=A, ld_t=64, t_dtype=3, w=A, w_dtype=3, offset=0.0, eps=1e-6, rows=4, H=64,
            y=A, ld_y=64, codes=A, ld_codes=64, scales=A, ld_s=4, rstd=A, stream=None)
NORM_BACK = dict(dy=A, ld_dy=64, total=A, ld_t=64, t_dtype=3, w=A, w_dtype=2, offset=0.0, rstd=A, dtotal=A, ld_dt=64, rows=4, H=64,
                 dx=A, ld_dx=64, dw=A, accumulate=0, ws=A, ws_bytes=1 << 20, stream=None)
DISPATCH = dict(x=A, ld_x=128, row_bytes=128, T=4, k=2, slot=A, P=8, count=A, out=A, ld_out=128, xs=A, ld_xs=4, blocks=1, os=A,
                ld_os=8, w=A, row_w=A, pos=A, stream=None)
DISPATCH_BACK = dict(dout=A, ld_d=64, d_dtype=3, pos=A, T=4, k=2, P=8, H=64, drow=A, dx=A, ld_dx=64, dx_dtype=2, dw=A, stream=None)
COMBINE = dict(y=A, ld_y=64, y_dtype=3, pos=A, w=A, T=4, k=2, P=8, H=64, add=A, ld_add=64, out=A, ld_out=64, out_dtype=3,
               stream=None)
COMBINE_BACK = dict(dout=A, ld_d=64, d_dtype=2, y=A, ld_y=64, y_dtype=3, pos=A, w=A, T=4, k=2, P=8, H=64, dy=A, ld_dy=64, dw=A,
                    stream=None)
PRODUCT = dict(x=A, ld_x=32, xs=A, ld_xs=8, w=A, wscale=A, offs=A, E=2, P=8, N=128, K=64, y=A, ld_y=128, dtype=3, ws=A,
               ws_bytes=256, stream=None)
QUANT = dict(src=A, dtype=3, ld=64, rows=4, K=64, codes=A, ld_codes=32, scales=A, ld_s=4, stream=None)
QUANT_W = dict(src=A, dtype=3, E=2, N=4, K=64, codes=A, tiles=A, stream=None)
PACK = dict(src=A, E=2, N=4, K=64, tiles=A, stream=None)
SWIGLU = dict(gu=A, ld_gu=128, w=A, rows=4, I=64, codes=A, ld_codes=32, scales=A, ld_s=4, stream=None)

CALLS = {"ft_moe_rmsnorm": NORM, "ft_moe_rmsnorm_backward": NORM_BACK, "ft_moe_dispatch": DISPATCH,
         "ft_moe_dispatch_backward": DISPATCH_BACK, "ft_moe_combine": COMBINE, "ft_moe_combine_backward": COMBINE_BACK,
         "ft_moe_group_gemm_mxfp4": PRODUCT, "ft_moe_quantize_mxfp4": QUANT, "ft_moe_quantize_mxfp4_weights": QUANT_W,
         "ft_moe_pack_mxfp4_scales": PACK, "ft_moe_swiglu_quantize_mxfp4": SWIGLU}

ORDER = [(dict(T=-1), 1), (dict(k=0), 1), (dict(P=-1), 1), (dict(k=33), 3), (dict(T=(1 << 20) + 1), 3), (dict(P=(1 << 25) + 1), 3)]
REFUSED = {
    "ft_moe_rmsnorm": [
        (dict(rows=-1), 1), (dict(H=0), 1), (dict(H=16385), 3), (dict(rows=(1 << 25) + 1), 3), (dict(eps=-1.0), 1),
        (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(offset=float("inf")), 1), (dict(H=40), 3),
        (dict(y=None, codes=None), 1), (dict(x=None), 1), (dict(x=A + 1), 1), (dict(ld_x=63), 1), (dict(residual=None), 1),
        (dict(total=None), 1), (dict(t_dtype=0), 1), (dict(t_dtype=2, total=A + 2), 1), (dict(ld_t=60), 1), (dict(ld_r=1), 1),
        (dict(w=None), 1), (dict(w_dtype=1), 1), (dict(w=A + 2, w_dtype=2), 1), (dict(y=A + 1), 1), (dict(ld_y=32), 1),
        (dict(codes=A + 8), 1), (dict(ld_codes=72), 1), (dict(scales=None), 1), (dict(ld_s=3), 1), (dict(rstd=A + 2), 1)],
    "ft_moe_rmsnorm_backward": [
        (dict(rows=-1), 1), (dict(H=-5), 1), (dict(H=20000), 3), (dict(offset=float("nan")), 1), (dict(accumulate=2), 1),
        (dict(dw=A + 1), 1), (dict(dy=None), 1), (dict(ld_dy=0), 1), (dict(total=A + 1), 1), (dict(t_dtype=7), 1), (dict(w=None), 1),
        (dict(rstd=None), 1), (dict(rstd=A + 2), 1), (dict(dtotal=A + 1), 1), (dict(ld_dt=63), 1), (dict(dx=None), 1),
        (dict(ld_dx=63), 1), (dict(ws=None), 1), (dict(ws=A + 16), 1), (dict(ws_bytes=64 * 4 - 1), 4)],
    "ft_moe_dispatch": ORDER + [
        (dict(row_bytes=0), 1), (dict(row_bytes=127), 1), (dict(row_bytes=262146), 3), (dict(blocks=-1), 1), (dict(blocks=513), 3),
        (dict(pos=A + 2), 1), (dict(slot=None), 1), (dict(slot=A + 1), 1), (dict(count=A + 2), 1), (dict(x=None), 1),
        (dict(x=A + 1), 1), (dict(ld_x=126), 1), (dict(ld_x=129), 1), (dict(out=None), 1), (dict(ld_out=64), 1), (dict(xs=None), 1),
        (dict(os=A + 2), 1), (dict(ld_xs=3), 1), (dict(ld_os=7), 1), (dict(w=None), 1), (dict(row_w=A + 1), 1)],
    "ft_moe_dispatch_backward": ORDER + [
        (dict(H=0), 1), (dict(H=65537), 3), (dict(dout=None), 1), (dict(d_dtype=0), 1), (dict(ld_d=63), 1), (dict(pos=None), 1),
        (dict(dx=A + 2), 1), (dict(dx_dtype=1), 1), (dict(ld_dx=3), 1), (dict(dw=A + 1), 1), (dict(drow=None), 1)],
    "ft_moe_combine": ORDER + [
        (dict(H=-1), 1), (dict(y=None), 1), (dict(y=A + 1), 1), (dict(y_dtype=9), 1), (dict(pos=A + 2), 1), (dict(w=A + 2), 1),
        (dict(add=A + 1), 1), (dict(ld_add=63), 1), (dict(out=None), 1), (dict(out_dtype=0), 1), (dict(ld_out=0), 1)],
    "ft_moe_combine_backward": ORDER + [
        (dict(H=0), 1), (dict(dout=A + 2), 1), (dict(d_dtype=0), 1), (dict(pos=None), 1), (dict(w=A + 2), 1), (dict(dw=A + 2), 1),
        (dict(y=None), 1), (dict(y_dtype=0), 1), (dict(dy=None), 1), (dict(ld_dy=63), 1)],
    "ft_moe_group_gemm_mxfp4": [
        (dict(E=0), 1), (dict(E=1025), 3), (dict(P=-1), 1), (dict(P=(1 << 25) + 1), 3), (dict(N=0), 1), (dict(K=-32), 1),
        (dict(N=65537), 3), (dict(K=65568), 3), (dict(K=48), 3), (dict(offs=None), 1), (dict(offs=A + 2), 1), (dict(dtype=0), 1),
        (dict(ws=None), 1), (dict(ws=A + 16), 1), (dict(ws_bytes=255), 4), (dict(x=None), 1), (dict(x=A + 8), 1), (dict(ld_x=40), 1),
        (dict(ld_x=16), 1), (dict(w=A + 8), 1), (dict(y=A + 2), 1), (dict(ld_y=127), 1), (dict(xs=None), 1), (dict(xs=A + 4), 1),
        (dict(ld_xs=10), 1), (dict(ld_xs=4), 1), (dict(wscale=None), 1), (dict(wscale=A + 8), 1)],
    "ft_moe_quantize_mxfp4": [
        (dict(dtype=0), 1), (dict(rows=-1), 1), (dict(K=0), 1), (dict(K=48), 3), (dict(src=None), 1), (dict(src=A + 8), 1),
        (dict(ld=60), 1), (dict(ld=68), 1), (dict(codes=A + 8), 1), (dict(ld_codes=40), 1), (dict(scales=None), 1), (dict(ld_s=3), 1)],
    "ft_moe_quantize_mxfp4_weights": [
        (dict(dtype=1), 1), (dict(E=0), 1), (dict(E=2000), 3), (dict(N=0), 1), (dict(K=16), 3), (dict(src=None), 1),
        (dict(codes=A + 4), 1), (dict(tiles=None), 1), (dict(tiles=A + 4), 1)],
    "ft_moe_pack_mxfp4_scales": [(dict(E=-1), 1), (dict(N=70000), 3), (dict(K=40), 3), (dict(src=None), 1), (dict(tiles=A + 8), 1)],
    "ft_moe_swiglu_quantize_mxfp4": [
        (dict(rows=-1), 1), (dict(I=48), 3), (dict(gu=A + 2), 1), (dict(ld_gu=132), 1), (dict(codes=None), 1),
        (dict(scales=A + 2), 1), (dict(w=A + 1), 1)],
}
CASES = [(n, c, code) for n, cases in REFUSED.items() for c, code in cases]


@pytest.mark.parametrize("name,change,code", CASES, ids=[f"{n[7:]}-{c}" for n, c, _ in CASES])
def test_refusals(ft, name, change, code):
    args = dict(CALLS[name], **change)
    assert getattr(ft.load(), name)(*args.values()) == code
    assert ft.ft_last_error()


@pytest.mark.parametrize("name,change", [
    ("ft_moe_rmsnorm", dict(rows=0, x=None, y=None, codes=None)), ("ft_moe_rmsnorm_backward", dict(rows=0, dy=None, dw=None)),
    ("ft_moe_rmsnorm_backward", dict(rows=0, accumulate=1)), ("ft_moe_dispatch", dict(P=0, pos=None, slot=None)),
    ("ft_moe_dispatch", dict(P=0, T=0)), ("ft_moe_dispatch_backward", dict(T=0, dx=None)), ("ft_moe_combine", dict(T=0, out=None)),
    ("ft_moe_combine_backward", dict(T=0, dout=None)), ("ft_moe_quantize_mxfp4", dict(rows=0, src=None)),
    ("ft_moe_swiglu_quantize_mxfp4", dict(rows=0, gu=None))])
def test_nothing_to_do_is_a_no_op(ft, name, change):
    assert getattr(ft.load(), name)(*dict(CALLS[name], **change).values()) == 0
    assert ft.ft_last_error() == ""


def test_workspace_size(ft):
    lib, n = ft.load(), ctypes.c_size_t()
    assert lib.ft_moe_rmsnorm_workspace_size(4, 64, None) == 1
    assert lib.ft_moe_rmsnorm_workspace_size(4, 0, ctypes.byref(n)) == 1
    assert lib.ft_moe_rmsnorm_workspace_size(4, 16385, ctypes.byref(n)) == 3
    assert ft.ft_moe_rmsnorm_workspace_size(0, 64) == 0
    assert ft.ft_moe_rmsnorm_workspace_size(1, 64) == 256
    assert ft.ft_moe_rmsnorm_workspace_size(1 << 25, 16384) <= 152 * 8 * 16384 * 4


def test_binding_refuses_what_it_cannot_pass(ft):
    """Types, shapes and layouts the C call cannot see; the last ones are well formed, but not on the GPU."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    f32, u8, i32 = torch.float32, torch.uint8, torch.int32
    x, w, slot, pos = z(4, 64), z(64), z(8, dtype=i32), z(4, 2, dtype=i32)
    c4, s4, w4, t4 = z(4, 32, dtype=u8), z(1, 4, 4, dtype=u8), z(2, 8, 32, dtype=u8), z(2, 1, 1, 512, dtype=u8)
    offs, ws, y = z(3, dtype=i32), z(256, dtype=u8), z(4, 8)
    bad = [
        lambda: ft.ft_moe_rmsnorm(x.float(), w, 1e-6, y=x),
        lambda: ft.ft_moe_rmsnorm(x, w[:32], 1e-6, y=x),
        lambda: ft.ft_moe_rmsnorm(x, w.half(), 1e-6, y=x),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, y=x.float()),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, y=x, residual=x),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, y=x, residual=x, total=x.float()),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, codes=x.byte()),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, codes=x.byte(), scales=z(4, 1, dtype=f32)),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, y=z(64, 4).t()),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, y=x, rstd=z(4)),
        lambda: ft.ft_moe_rmsnorm_backward(x, x, w, z(4, dtype=f32), x.float()),
        lambda: ft.ft_moe_rmsnorm_backward(x, x, w, z(4, dtype=f32), x, dw=w),
        lambda: ft.ft_moe_rmsnorm_backward(x, x, w, z(3, dtype=f32), x),
        lambda: ft.ft_moe_rmsnorm_backward(x, x, w, z(4, dtype=f32), x, dtotal=x.float()),
        lambda: ft.ft_moe_dispatch(x, slot.long(), 2, z(8, 64)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64, dtype=f32)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(7, 64)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64), x_scale=z(1, 4, dtype=f32)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64), x_scale=z(1, 4, dtype=f32), out_scale=z(1, 7, dtype=f32)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64), x_scale=s4, out_scale=z(1, 8, dtype=f32)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64), w=z(4, 2, dtype=f32)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64), w=z(4, 3, dtype=f32), row_w=z(8, dtype=f32)),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64), pos=z(8, dtype=i32)),
        lambda: ft.ft_moe_dispatch_backward(z(8, 64), pos, x, dw=z(4, 2, dtype=f32)),
        lambda: ft.ft_moe_dispatch_backward(z(8, 64), pos, z(4, 32)),
        lambda: ft.ft_moe_combine(z(8, 64), pos, z(4, 2), x),
        lambda: ft.ft_moe_combine(z(8, 64), pos, None, x, add=x.float()),
        lambda: ft.ft_moe_combine(z(8, 64).half(), pos, None, x),
        lambda: ft.ft_moe_combine_backward(x, None, pos, None, z(8, 64), dw=z(4, 2, dtype=f32)),
        lambda: ft.ft_moe_combine_backward(x, z(8, 32), pos, None, z(8, 64)),
        lambda: ft.ft_moe_combine_backward(x, None, pos, None, z(8, 64, dtype=f32)),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4.view(torch.int8), s4, w4, t4, offs, y, ws),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, s4[:, :3], w4, t4, offs, y, ws),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, s4[:, :, :2], w4, t4, offs, y, ws),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, z(1, 4, 8, dtype=u8)[:, :, ::2], w4, t4, offs, y, ws),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, s4, w4, t4[:1], offs, y, ws),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, s4, w4.transpose(1, 2).contiguous().transpose(1, 2), t4, offs, y, ws),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, s4, w4, t4, None, y, ws),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, s4, w4, t4, offs, y.half(), ws),
        lambda: ft.ft_moe_quantize_mxfp4(x, c4[:, :16], s4),
        lambda: ft.ft_moe_quantize_mxfp4(x.half(), c4, s4),
        lambda: ft.ft_moe_quantize_mxfp4_weights(z(2, 8, 64), w4, t4[:, :, :, :256]),
        lambda: ft.ft_moe_pack_mxfp4_scales(z(2, 8, 2, dtype=f32), t4),
        lambda: ft.ft_moe_swiglu_quantize_mxfp4(z(4, 64), None, c4, s4),
        lambda: ft.ft_moe_rmsnorm(x, w, 1e-6, y=x),
        lambda: ft.ft_moe_dispatch(x, slot, 2, z(8, 64)),
        lambda: ft.ft_moe_combine(z(8, 64), pos, None, x),
        lambda: ft.ft_moe_group_gemm_mxfp4(c4, s4, w4, t4, offs, y, ws),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)


def test_plan_refusals(ft):
    plan = (ctypes.c_int32 * 4)()
    call = ft.load().ft_moe_debug_group_plan
    good = dict(product=4, E=2, P=8, N=128, K=64, dtype=2, accumulate=0, plan=plan)
    for change, code in ((dict(product=5), 1), (dict(P=0), 1), (dict(plan=None), 1), (dict(accumulate=1), 1), (dict(dtype=0), 1),
                         (dict(K=48), 3), (dict(E=1025), 3)):
        assert call(*dict(good, **change).values()) == code, change
        assert ft.ft_last_error()
