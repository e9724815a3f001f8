"""A routed expert layer on 16-bit weights, trained for a few steps, and the
same layer served from E4M3 weights with one scale per block of 128.

    python examples/expert_layer.py

Router -> permute -> gate/up product -> SiTU -> down product -> weighted sum,
plus a shared expert when serving.  Everything between the products is plain
torch; the routing, the permute, the products, their gradients and the
quantisation are the library's.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from block_scaled_fp4_permute_gb300 import binding as b  # noqa: E402


def situ(gate_up, beta=1.0, beta_lin=0.0):
    """b tanh(g / b) sigmoid(g) * (bl tanh(u / bl), or u where bl is 0), in fp32."""
    g, u = gate_up.float().chunk(2, dim=-1)
    if beta_lin > 0:
        u = beta_lin * torch.tanh(u / beta_lin)
    return beta * torch.tanh(g / beta) * torch.sigmoid(g) * u


def route(x, router, top_k):
    """(slots' rows sorted by expert, their tokens, their weights, offsets)."""
    ids, weights = b.situ_moe_route_topk(x.detach().float() @ router.T, top_k)
    experts = router.shape[0]
    _, offsets, slot, _ = b.situ_moe_permute(ids, experts, experts, 0)
    slot = slot.long()
    return slot // top_k, weights.reshape(-1)[slot], offsets


def forward(x, router, w1, w2, top_k):
    """The layer on 16-bit weights, differentiable in x, w1 and w2: x [T, H],
    w1 [E, 2I, H], w2 [E, H, I]."""
    token, weight, offsets = route(x, router, top_k)
    h = situ(b.grouped_linear(x[token], w1, offsets)).to(x.dtype)
    y = b.grouped_linear(h, w2, offsets)
    return torch.zeros(x.shape, device=x.device).index_add(0, token, y.float() * weight[:, None])


class Fp8Layer:
    """The layer for serving: weights quantised once, activations per call."""

    def __init__(self, router, w1, w2, shared1, shared2, top_k):
        self.router, self.top_k = router, top_k
        self.w1, self.w2 = b.situ_moe_quant_fp8(w1, 128), b.situ_moe_quant_fp8(w2, 128)
        self.shared1, self.shared2 = b.situ_moe_quant_fp8(shared1, 128), b.situ_moe_quant_fp8(shared2, 128)

    def __call__(self, x):
        token, weight, offsets = route(x, self.router, self.top_k)
        q, scale = b.situ_moe_quant_fp8(x)                       # once per token, not per slot
        h = situ(b.situ_moe_fp8_grouped_gemm(q[token], scale[token], *self.w1, offsets))
        y = b.situ_moe_fp8_grouped_gemm(*b.situ_moe_quant_fp8(h), *self.w2, offsets, out_dtype=torch.float32)
        hs = situ(b.situ_moe_fp8_gemm(q, scale, *self.shared1))
        out = b.situ_moe_fp8_gemm(*b.situ_moe_quant_fp8(hs), *self.shared2, out_dtype=torch.float32)
        return out.index_add(0, token, y * weight[:, None])


def main(T=256, H=512, I=256, E=16, top_k=4, steps=20, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std):
        return torch.randn(shape, generator=g, device=device) * std

    x = normal(T, H, std=1.0).bfloat16()
    router = normal(E, H, std=H ** -0.5)
    target = normal(T, H, std=0.5)
    w1 = normal(E, 2 * I, H, std=H ** -0.5).bfloat16().requires_grad_()
    w2 = normal(E, H, I, std=I ** -0.5).bfloat16().requires_grad_()
    losses = []
    master = [w.detach().float() for w in (w1, w2)]               # updates in fp32, products in bf16
    for _ in range(steps):
        w1.grad = w2.grad = None
        loss = (forward(x, router, w1, w2, top_k) - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for w, m in zip((w1, w2), master):
                m -= 0.02 * w.grad.float() / w.grad.float().square().mean().sqrt().clamp(min=1e-12) * m.square().mean().sqrt()
                w.copy_(m)
        losses.append(loss.item())
    zeros = torch.zeros(2 * I, H, device=device), torch.zeros(H, I, device=device)
    served = Fp8Layer(router, w1.detach(), w2.detach(), *zeros, top_k)(x)
    trained = forward(x, router, w1, w2, top_k).detach()
    off = ((served - trained).norm() / trained.norm()).item()
    if b.situ_moe_gemm_status() != 0:
        raise RuntimeError("a kernel gave up a wait")
    return losses, off


if __name__ == "__main__":
    losses, off = main()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    print(f"served from E4M3 weights: {100 * off:.1f} % off the 16-bit layer (2-norm)")
