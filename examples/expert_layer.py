"""A routed expert layer from the library's parts: a training step on bf16 weights, and a serving
step on 8-bit weights (fp8_block banks as ft_moe_pack fills them).

    route -> align -> gather -> product -> SwiGLU -> product -> combine

Training runs the products, their gradients and SwiGLU's backward through the library and lets
torch differentiate the rest (the router's softmax, the loss). Serving quantizes the tokens once,
multiplies 8-bit rows with 8-bit weights and stores the SwiGLU result in 8 bits.

    python examples/expert_layer.py        # needs the built library and a GB300
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_quantized_moe_gb300 as ft  # noqa: E402


class Plan:
    """Where each of the T * k slots goes: rows sorted by expert (no padding), and back."""

    def __init__(self, ids: torch.Tensor, E: int):
        T, k = ids.shape
        dev = ids.device
        n = T * k
        self.T, self.k, self.rows = T, k, n
        self.slot = torch.empty(n, dtype=torch.int32, device=dev)
        block, self.offs = torch.empty(n + 1, dtype=torch.int32, device=dev), torch.empty(E + 1, dtype=torch.int32, device=dev)
        count = torch.empty(1, dtype=torch.int32, device=dev)
        ws = torch.empty(ft.ft_moe_align_workspace_size(T, k, E), dtype=torch.uint8, device=dev)
        ft.ft_moe_align(ids, E, 1, self.slot, block, self.offs, count, ws)
        self.slot = self.slot.long()
        self.token = self.slot // k
        self.back = torch.empty_like(self.slot)
        self.back[self.slot] = torch.arange(n, device=dev)

    def combine(self, y: torch.Tensor) -> torch.Tensor:
        """Sum of each token's rows, in the order of its slots."""
        return y[self.back].view(self.T, self.k, -1).float().sum(1)


def route(logits: torch.Tensor, k: int):
    """Expert ids and weights of fp32 logits [T, E]."""
    ids = torch.empty((logits.shape[0], k), dtype=torch.int32, device=logits.device)
    w = torch.empty((logits.shape[0], k), dtype=torch.float32, device=logits.device)
    ft.ft_moe_route(logits, k, ids, w)
    return ids, w


def _workspace(E, P, N, K, device):
    return torch.empty(ft.ft_moe_group_workspace_size(E, P, N, K), dtype=torch.uint8, device=device)


class Experts(torch.autograd.Function):
    """out[t] = sum over t's slots of w_row * down_e(silu(gate_e x) * up_e x), with all gradients.
    x bf16 [T, H], row weights fp32 [T * k] (sorted order), w_gate_up bf16 [E, 2 I, H], w_down bf16 [E, H, I]."""

    @staticmethod
    def forward(ctx, x, row_w, w_gate_up, w_down, plan):
        E, I2, H = w_gate_up.shape
        P, I, dev = plan.rows, I2 // 2, x.device
        ws = _workspace(E, P, max(I2, H), max(I2, H), dev)
        xs = x[plan.token]
        gu = torch.empty((P, I2), dtype=torch.bfloat16, device=dev)
        h = torch.empty((P, I), dtype=torch.bfloat16, device=dev)
        y = torch.empty((P, H), dtype=torch.float32, device=dev)
        ft.ft_moe_group_gemm(xs, w_gate_up, plan.offs, gu, ws)
        ft.ft_moe_swiglu(gu, row_w, h)
        ft.ft_moe_group_gemm(h, w_down, plan.offs, y, ws)
        ctx.plan, ctx.ws = plan, ws
        ctx.save_for_backward(xs, row_w, gu, h, w_gate_up, w_down)
        return plan.combine(y)

    @staticmethod
    def backward(ctx, dout):
        xs, row_w, gu, h, w_gate_up, w_down = ctx.saved_tensors
        plan, ws = ctx.plan, ctx.ws
        dy = dout.bfloat16()[plan.token]
        dh, dgu = torch.empty_like(h), torch.empty_like(gu)
        drow = torch.empty_like(row_w)
        dxs = torch.empty((plan.rows, xs.shape[1]), dtype=torch.float32, device=xs.device)
        dw_down = torch.empty(w_down.shape, dtype=torch.float32, device=xs.device)
        dw_gate_up = torch.empty(w_gate_up.shape, dtype=torch.float32, device=xs.device)
        ft.ft_moe_group_gemm_dgrad(dy, w_down, plan.offs, dh, ws)
        ft.ft_moe_group_gemm_wgrad(dy, h, plan.offs, dw_down, ws)
        ft.ft_moe_swiglu_backward(gu, row_w, dh, dgu, drow)
        ft.ft_moe_group_gemm_dgrad(dgu, w_gate_up, plan.offs, dxs, ws)
        ft.ft_moe_group_gemm_wgrad(dgu, xs, plan.offs, dw_gate_up, ws)
        return plan.combine(dxs).to(xs.dtype), drow, dw_gate_up, dw_down, None


def train_forward(x, w_router, w_gate_up, w_down, k):
    """Layer output fp32 [T, H], differentiable in x and every weight (w_router fp32 [E, H])."""
    logits = x.float() @ w_router.t()
    ids, _ = route(logits.detach().contiguous(), k)
    plan = Plan(ids, w_gate_up.shape[0])
    kept = torch.softmax(logits, 1).gather(1, ids.long())
    weights = kept / kept.sum(1, keepdim=True)
    return Experts.apply(x, weights.reshape(-1)[plan.slot].contiguous(), w_gate_up, w_down, plan)


def serve_forward(x, ids, weights, gate_up, gate_up_scale, down, down_scale):
    """Layer output fp32 [T, H] on 8-bit banks: gate_up u8 [E, 2 I, H] with scales [E, 2 I / 128, H / 128],
    down u8 [E, H, I] with scales [E, H / 128, I / 128]."""
    E, I2, H = gate_up.shape
    T, I, dev = x.shape[0], I2 // 2, x.device
    plan = Plan(ids, E)
    P = plan.rows
    ws = _workspace(E, P, max(I2, H), max(I2, H), dev)
    codes = torch.empty((T, H), dtype=torch.uint8, device=dev)
    scales = torch.empty((H // 128, T), dtype=torch.float32, device=dev)
    ft.ft_moe_quantize_fp8(x, codes, scales)
    gu = torch.empty((P, I2), dtype=torch.bfloat16, device=dev)
    ft.ft_moe_group_gemm_fp8(codes[plan.token], scales[:, plan.token].contiguous(), gate_up, gate_up_scale, plan.offs, gu, ws)
    hc = torch.empty((P, I), dtype=torch.uint8, device=dev)
    hs = torch.empty((I // 128, P), dtype=torch.float32, device=dev)
    ft.ft_moe_swiglu_quantize_fp8(gu, weights.reshape(-1)[plan.slot].contiguous(), hc, hs)
    y = torch.empty((P, H), dtype=torch.float32, device=dev)
    ft.ft_moe_group_gemm_fp8(hc, hs, down, down_scale, plan.offs, y, ws)
    return plan.combine(y)


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
