"""The example layer: its forward and gradients against plain fp32 torch, the
training loop's progress, and the E4M3 form's distance from the 16-bit one."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from block_scaled_fp4_permute_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    build.build()
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_layer_and_gradients_match_plain_torch(ex):
    T, H, I, E, K = 60, 128, 64, 6, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16().requires_grad_()
    router = torch.randn((E, H), generator=g, device="cuda") * H ** -0.5
    w1 = (torch.randn((E, 2 * I, H), generator=g, device="cuda") * H ** -0.5).bfloat16().requires_grad_()
    w2 = (torch.randn((E, H, I), generator=g, device="cuda") * I ** -0.5).bfloat16().requires_grad_()
    out = ex.forward(x, router, w1, w2, K)
    dout = torch.randn((T, H), generator=g, device="cuda")
    out.backward(dout)

    xd, w1d, w2d = (t.detach().double().requires_grad_() for t in (x, w1, w2))
    logits = x.detach().float() @ router.T
    top, ids = logits.topk(K, dim=1)
    weight = torch.softmax(top.double(), dim=1)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for k in range(K):
        gate_up = torch.einsum("th,tnh->tn", xd, w1d[ids[:, k]])
        gg, u = gate_up.chunk(2, dim=-1)
        h = torch.tanh(gg) * torch.sigmoid(gg) * u
        ref = ref + weight[:, k:k + 1] * torch.einsum("ti,thi->th", h, w2d[ids[:, k]])
    ref.backward(dout.double())
    # bf16 roundings of the gate/up product, the activation, the down product
    # and, backwards, of each gradient: up to six of 2^-8 each, and their
    # products through factors of order one: 2^-4 of the norm bounds them
    for got, want in ((out, ref), (x.grad, xd.grad), (w1.grad, w1d.grad), (w2.grad, w2d.grad)):
        assert ((got.double() - want).norm() <= 2.0 ** -4 * want.norm()).item()


def test_example_trains_and_serves(ex):
    losses, off = ex.main(T=128, H=256, I=128, E=8, top_k=2, steps=10)
    assert losses[-1] < losses[0] and all(v == v for v in losses)
    # four E4M3 factors per product chain, 2^-4 relative each
    assert off <= 4 * 2.0 ** -4
