"""Fine-tuning a routed expert layer, and serving what came of it.

    python examples/expert_finetune.py

The router and the experts are trained with a balance loss, the experts' inputs
kept in 8 bits for the backward pass, beside one low-rank adapter per expert.
Then a shared projection on E4M3 weights serves a batch in which every request
has an adapter of its own, or none.  Everything between the calls is plain torch.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from block_scaled_fp4_permute_gb300 import binding as b  # noqa: E402


def forward(x, p, top_k, coef=0.01, mask=None, keep="mxfp8"):
    """(layer output fp32 [T, H], slots per expert, balance loss): x [T, H] in 16
    bits, p a dict of the router [E, H] (fp32), w1 [E, 2I, H], w2 [E, H, I], the
    caps p0 and p1 [E], and adapters a [E, r, H] and b [E, H, r] from a slot's
    input to its output.  Differentiable in x and all of these but the caps."""
    experts = p["router"].shape[0]
    ids, weights, counts, loss = b.balanced_route(x.float() @ p["router"].T, top_k, mask=mask, coef=coef)
    _, offsets, slot, _ = b.situ_moe_permute(ids, experts, experts, 0)
    slot = slot.long()
    rows = x[slot // top_k]
    y = b.expert_ffn(rows, p["w1"], p["w2"], offsets, p["p0"], p["p1"], keep=keep)
    y = b.lora_linear(y, rows, p["a"], p["b"], offsets)
    out = torch.zeros(x.shape, device=x.device).index_add(0, slot // top_k, y.float() * weights.reshape(-1)[slot, None])
    return out, counts, loss


class Projection:
    """A projection served to many requests: E4M3 weights, an adapter per request."""

    def __init__(self, w, a, b_):
        self.w, self.a, self.b = b.situ_moe_quant_fp8(w, 128), a, b_

    def __call__(self, x, ids, scale=None):
        base = b.situ_moe_fp8_gemm(*b.situ_moe_quant_fp8(x), *self.w)
        return b.situ_moe_lora(base, x, self.a, self.b, ids=ids, scale=scale, out=base)


def parameters(H, I, E, r, g, device="cuda"):
    def normal(*shape, std):
        return torch.randn(shape, generator=g, device=device) * std

    p = dict(router=normal(E, H, std=H ** -0.5), w1=normal(E, 2 * I, H, std=H ** -0.5).bfloat16(),
             w2=normal(E, H, I, std=I ** -0.5).bfloat16(), a=normal(E, r, H, std=H ** -0.5).bfloat16(),
             b=torch.zeros(E, H, r, device=device, dtype=torch.bfloat16))
    for t in p.values():
        t.requires_grad_()
    return dict(p, p0=torch.full((E,), 2.0, device=device), p1=torch.full((E,), 2.0, device=device))


def main(T=256, H=512, I=256, E=16, r=16, top_k=4, steps=20, requests=64, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn((T, H), generator=g, device=device).bfloat16()
    target = torch.randn((T, H), generator=g, device=device) * 0.5
    p = parameters(H, I, E, r, g, device)
    trained = [t for t in p.values() if t.requires_grad]
    master = [t.detach().float() for t in trained]                # updates in fp32, products in bf16
    losses, shares = [], []
    for _ in range(steps):
        for t in trained:
            t.grad = None
        out, counts, balance = forward(x, p, top_k)
        loss = (out - target).square().mean()
        (loss + balance).backward()
        with torch.no_grad():
            for t, m in zip(trained, master):
                m -= 0.02 * t.grad.float() / t.grad.float().square().mean().sqrt().clamp(min=1e-12) * H ** -0.5
                t.copy_(m)
        losses.append(loss.item())
        shares.append(counts.max().item() / (T * top_k))
    # the adapters that were trained, one to a request, on a projection of their sizes
    ids = torch.randint(-1, E, (requests,), generator=g, device=device).int()
    w = torch.randn((H, H), generator=g, device=device).bfloat16() * H ** -0.5
    served = Projection(w, p["a"].detach(), p["b"].detach())(x[:requests], ids)
    if b.situ_moe_gemm_status() != 0:
        raise RuntimeError("a kernel gave up a wait")
    return losses, shares, served


if __name__ == "__main__":
    losses, shares, served = main()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps, "
          f"the busiest expert's share of the slots {100 * shares[0]:.1f} -> {100 * shares[-1]:.1f} %")
    print(f"served {served.shape[0]} requests, each with an adapter of its own or none")
