"""A routed expert layer from the library's parts: a training step on bf16 weights, and serving steps on 8-bit weights
(fp8_block banks as ft_moe_pack fills them) and on 4-bit ones (MXFP4).

    (norm ->) route -> align -> dispatch -> product -> SwiGLU -> product -> combine

Training runs all of these and their gradients through the library and lets torch differentiate the rest (the
router's softmax, the loss). Serving quantizes the tokens once, multiplies 8-bit or 4-bit rows with weights of
the same kind and stores the SwiGLU result in that kind too.

    python examples/expert_layer.py        # needs the built library and a GB300
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_quantized_moe_gb300 as ft  # noqa: E402


class Plan:
    """Where each of the T * k slots goes: rows sorted by expert (no padding). pos, the way back, comes from the dispatch."""

    def __init__(self, ids: torch.Tensor, E: int):
        T, k = ids.shape
        dev = ids.device
        n = T * k
        self.T, self.k, self.rows = T, k, n
        self.slot, self.pos = torch.empty(n, dtype=torch.int32, device=dev), torch.empty((T, k), dtype=torch.int32, device=dev)
        block, self.offs = torch.empty(n + 1, dtype=torch.int32, device=dev), torch.empty(E + 1, dtype=torch.int32, device=dev)
        count = torch.empty(1, dtype=torch.int32, device=dev)
        ws = torch.empty(ft.ft_moe_align_workspace_size(T, k, E), dtype=torch.uint8, device=dev)
        ft.ft_moe_align(ids, E, 1, self.slot, block, self.offs, count, ws)


def route(logits: torch.Tensor, k: int):
    """Expert ids and weights of fp32 logits [T, E]."""
    ids = torch.empty((logits.shape[0], k), dtype=torch.int32, device=logits.device)
    w = torch.empty((logits.shape[0], k), dtype=torch.float32, device=logits.device)
    ft.ft_moe_route(logits, k, ids, w)
    return ids, w


def _workspace(E, P, N, K, device):
    return torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device=device)


class Experts(torch.autograd.Function):
    """out[t] = sum over t's slots of w[t, j] * down_e(silu(gate_e x) * up_e x), with all gradients.
    x bf16 [T, H], weights fp32 [T, k], w_gate_up bf16 [E, 2 I, H], w_down bf16 [E, H, I]."""

    @staticmethod
    def forward(ctx, x, weights, w_gate_up, w_down, plan):
        E, I2, H = w_gate_up.shape
        P, I, dev = plan.rows, I2 // 2, x.device
        ws = _workspace(E, P, max(I2, H), max(I2, H), dev)
        xs, row_w = torch.empty((P, H), dtype=x.dtype, device=dev), torch.empty(P, dtype=torch.float32, device=dev)
        gu = torch.empty((P, I2), dtype=torch.bfloat16, device=dev)
        h = torch.empty((P, I), dtype=torch.bfloat16, device=dev)
        y = torch.empty((P, H), dtype=torch.float32, device=dev)
        out = torch.empty((plan.T, H), dtype=torch.float32, device=dev)
        ft.ft_moe_dispatch(x, plan.slot, plan.k, xs, w=weights, row_w=row_w, pos=plan.pos)
        ft.ft_moe_group_gemm(xs, w_gate_up, plan.offs, gu, ws)
        ft.ft_moe_swiglu(gu, row_w, h)
        ft.ft_moe_group_gemm(h, w_down, plan.offs, y, ws)
        ft.ft_moe_combine(y, plan.pos, None, out)
        ctx.plan, ctx.ws = plan, ws
        ctx.save_for_backward(xs, row_w, gu, h, w_gate_up, w_down)
        return out

    @staticmethod
    def backward(ctx, dout):
        xs, row_w, gu, h, w_gate_up, w_down = ctx.saved_tensors
        plan, ws = ctx.plan, ctx.ws
        (P, H), dev = xs.shape, xs.device
        dy, dh, dgu = torch.empty_like(xs), torch.empty_like(h), torch.empty_like(gu)
        drow = torch.empty_like(row_w)
        dxs = torch.empty((P, H), dtype=torch.float32, device=dev)
        dx, dweights = torch.empty((plan.T, H), dtype=xs.dtype, device=dev), torch.empty((plan.T, plan.k), device=dev)
        dw_down = torch.empty(w_down.shape, dtype=torch.float32, device=dev)
        dw_gate_up = torch.empty(w_gate_up.shape, dtype=torch.float32, device=dev)
        ft.ft_moe_combine_backward(dout.contiguous(), None, plan.pos, None, dy)
        ft.ft_moe_group_gemm_dgrad(dy, w_down, plan.offs, dh, ws)
        ft.ft_moe_group_gemm_wgrad(dy, h, plan.offs, dw_down, ws)
        ft.ft_moe_swiglu_backward(gu, row_w, dh, dgu, drow)
        ft.ft_moe_group_gemm_dgrad(dgu, w_gate_up, plan.offs, dxs, ws)
        ft.ft_moe_group_gemm_wgrad(dgu, xs, plan.offs, dw_gate_up, ws)
        ft.ft_moe_dispatch_backward(dxs, plan.pos, dx, drow_w=drow, dw=dweights)
        return dx, dweights, dw_gate_up, dw_down, None


def train_forward(x, w_router, w_gate_up, w_down, k):
    """Layer output fp32 [T, H], differentiable in x and every weight (w_router fp32 [E, H])."""
    logits = x.float() @ w_router.t()
    ids, _ = route(logits.detach().contiguous(), k)
    plan = Plan(ids, w_gate_up.shape[0])
    kept = torch.softmax(logits, 1).gather(1, ids.long())
    weights = kept / kept.sum(1, keepdim=True)
    return Experts.apply(x, weights, w_gate_up, w_down, plan)


class Norm(torch.autograd.Function):
    """total = x + residual and y = total / rms(total) * weight, with all gradients (x and y bf16, total of residual's type,
    weight fp32 [H])."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        total, y = torch.empty_like(residual), torch.empty_like(x)
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        ft.ft_moe_rmsnorm(x, weight, eps, y=y, residual=residual, total=total, rstd=rstd)
        ctx.save_for_backward(total, weight, rstd)
        return total, y

    @staticmethod
    def backward(ctx, dtotal, dy):
        total, weight, rstd = ctx.saved_tensors
        dx, dw = torch.empty_like(total), torch.empty_like(weight)
        ws = torch.empty(ft.ft_moe_rmsnorm_workspace_size(*total.shape), dtype=torch.uint8, device=total.device)
        ft.ft_moe_rmsnorm_backward(dy.contiguous(), total, weight, rstd, dx, ws, dw=dw, dtotal=dtotal.contiguous())
        return dx.bfloat16(), dx, dw, None


def train_block(x, residual, w_norm, w_router, w_gate_up, w_down, k, eps=1e-6):
    """A residual block: x (bf16, the block before's output) joins the residual stream, whose norm goes through the expert
    layer. Returns the layer's output and the stream, for the next block's norm."""
    total, y = Norm.apply(x, residual, w_norm, eps)
    return train_forward(y, w_router, w_gate_up, w_down, k), total


def serve_forward(x, ids, weights, gate_up, gate_up_scale, down, down_scale):
    """Layer output fp32 [T, H] on 8-bit banks: gate_up u8 [E, 2 I, H] with scales [E, 2 I / 128, H / 128],
    down u8 [E, H, I] with scales [E, H / 128, I / 128]."""
    E, I2, H = gate_up.shape
    T, I, dev = x.shape[0], I2 // 2, x.device
    plan = Plan(ids, E)
    P = plan.rows
    ws = _workspace(E, P, max(I2, H), max(I2, H), dev)
    codes, scales = torch.empty((T, H), dtype=torch.uint8, device=dev), torch.empty((H // 128, T), device=dev)
    xc, xs, row_w = torch.empty((P, H), dtype=torch.uint8, device=dev), torch.empty((H // 128, P), device=dev), torch.empty(P, device=dev)
    gu = torch.empty((P, I2), dtype=torch.bfloat16, device=dev)
    hc, hs = torch.empty((P, I), dtype=torch.uint8, device=dev), torch.empty((I // 128, P), device=dev)
    y, out = torch.empty((P, H), device=dev), torch.empty((T, H), device=dev)
    ft.ft_moe_quantize_fp8(x, codes, scales)
    ft.ft_moe_dispatch(codes, plan.slot, plan.k, xc, x_scale=scales, out_scale=xs, w=weights, row_w=row_w, pos=plan.pos)
    ft.ft_moe_group_gemm_fp8(xc, xs, gate_up, gate_up_scale, plan.offs, gu, ws)
    ft.ft_moe_swiglu_quantize_fp8(gu, row_w, hc, hs)
    ft.ft_moe_group_gemm_fp8(hc, hs, down, down_scale, plan.offs, y, ws)
    ft.ft_moe_combine(y, plan.pos, None, out)
    return out


def serve_forward_mxfp4(x, ids, weights, gate_up, gate_up_tiles, down, down_tiles, shared=None):
    """The same on MXFP4 weights: gate_up u8 [E, 2 I, H / 2] and down u8 [E, H, I / 2] with their scale tiles, as
    ft_moe_quantize_mxfp4_weights makes them; the routing weights are applied on the way back. shared: fp32 [T, H] added."""
    (E, I2, half), H = gate_up.shape, down.shape[1]
    T, I, dev = x.shape[0], I2 // 2, x.device
    plan = Plan(ids, E)
    P = plan.rows
    ws = _workspace(E, P, max(I2, H), max(I2, H), dev)
    codes, scales = torch.empty((T, half), dtype=torch.uint8, device=dev), ft.alloc_mxfp4_scales(T, H, dev)
    xc, xs = torch.empty((P, half), dtype=torch.uint8, device=dev), ft.alloc_mxfp4_scales(P, H, dev)
    gu = torch.empty((P, I2), dtype=torch.bfloat16, device=dev)
    hc, hs = torch.empty((P, I // 2), dtype=torch.uint8, device=dev), ft.alloc_mxfp4_scales(P, I, dev)
    y, out = torch.empty((P, H), dtype=torch.bfloat16, device=dev), torch.empty((T, H), device=dev)
    ft.ft_moe_quantize_mxfp4(x, codes, scales)
    ft.ft_moe_dispatch(codes, plan.slot, plan.k, xc, x_scale=scales, out_scale=xs, pos=plan.pos)
    ft.ft_moe_group_gemm_mxfp4(xc, xs, gate_up, gate_up_tiles, plan.offs, gu, ws)
    ft.ft_moe_swiglu_quantize_mxfp4(gu, None, hc, hs)
    ft.ft_moe_group_gemm_mxfp4(hc, hs, down, down_tiles, plan.offs, y, ws)
    ft.ft_moe_combine(y, plan.pos, weights, out, add=shared)
    return out


def main(T: int = 2048, H: int = 2048, I: int = 512, E: int = 64, k: int = 8, steps: int = 5) -> list[float]:
    """A few steps of gradient descent towards a fixed target; returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(0)

    def weight(*shape):
        return torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5

    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    target = torch.randn((T, H), generator=gen, device="cuda") * 0.1
    master = [weight(E, H), weight(E, 2 * I, H), weight(E, H, I)]  # router, gate_up, down
    losses = []
    for _ in range(steps):
        live = [master[0].requires_grad_(), *(m.bfloat16().requires_grad_() for m in master[1:])]
        loss = ((train_forward(x, *live, k) - target) ** 2).sum() / T
        grads = torch.autograd.grad(loss, live)
        with torch.no_grad():
            master = [(m - 0.02 * g.float()).detach() for m, g in zip(master, grads)]
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    for step, loss in enumerate(main()):
        print(f"step {step}: loss {loss:.4f}")
