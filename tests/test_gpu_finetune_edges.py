"""The fine-tuning operators far from ordinary values, against plain
implementations in 64 bits.  H, U: half an ulp of a 16-bit type and of fp32."""
import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build
from test_gpu_finetune import BF16, F16, F32, H, TINY, U, gen, normal, offsets_of, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()
    yield
    assert B.situ_moe_gemm_status() == 0


# --------------------------------------------------------------------------
# gradients of f16 adapters
# --------------------------------------------------------------------------

def gradients(dy, x, a, b, counts, scale):
    """Per adapter (p, |p|'s sums, its other factor) of dA = p^T t and dB = (p^T t)^T in 64 bits."""
    at = 0
    for e, n in enumerate(counts):
        rows = slice(at, at + n)
        at += n
        f, ae, be, xe, de = scale[e].double(), a[e].double(), b[e].double(), x[rows].double(), dy[rows].double()
        yield e, (f * (de @ be), f * (de.abs() @ be.abs()), xe), (f * (xe @ ae.T), f * (xe.abs() @ ae.abs().T), de)


# A sum p^T t over L rows: p itself a sum of C terms (2 (C + 40) U of their magnitudes), taken in two terms of f16 under
# a power of two that brings the adapter's largest to [2^14, 2^15): off by 2^-22 relative, or half a subnormal's step,
# 2^-25 beside 2^14.  A row of u that the forward pass's terms hold (its largest 2^-8 or more, below 2^16) is off by
# half of f16's smallest step, 2^-25, instead.  The sum truncates 2 U a row; the result's rounding, and a tenth of it
# more for long sums.
def far_bar(want, p, pa, t, C, kept=False):
    most = p.abs().max() if p.numel() else 0.0
    largest = p.abs().amax(1) if p.numel() else p.sum(1)
    held = kept & (largest >= 2.0 ** -8.1) & (largest < 2.0 ** 16)
    return (1.1 * H[F16] * want.abs() + (2.0 ** -22 + 2 * len(p) * U) * (p.abs().T @ t.abs())
            + 2.0 ** -39 * most * t.abs().sum(0)[None] + 2.0 ** -25 * t[held].abs().sum(0)[None]
            + (2 * C + 80) * U * (pa.T @ t.abs()) + TINY[F16] / 2)


@pytest.mark.parametrize("dy_std,b_std,x_std,a_std,f", [
    (1e-3, 1e-3, 30.0, 0.05, 1.0), (1e-4, 1e-4, 1e3, 1e-3, 1.0), (1e-4, 1e-5, 5e3, 1e-2, 1.0),     # v of 5e-5 to 5e-8
    (2e-3, 1e-6, 1e4, 1e-3, 2.0 ** -9), (1e3, 30.0, 1e-4, 1.0, 1.0),                                # v of 1e-10 and of 1e6
    (3e-5, 1e-2, 30.0, 3e3, 1.0), (1e-6, 1.0, 300.0, 1e4, 1.0),                                     # u of 2^21 and 2^26
    (100.0, 1e-3, 1e-3, 1e-3, 1.0), (1e3, 1e-3, 1e-5, 1e-5, 2.0 ** -6)])                            # u of 2^-15 and 2^-36
@pytest.mark.parametrize("counts,K,N,r", [([300, 0, 77], 520, 264, 16), ([1500], 1032, 520, 64)])
def test_f16_gradients_far_from_one(dy_std, b_std, x_std, a_std, f, counts, K, N, r):
    g = gen(K)
    S, n, off = sum(counts) + 3, len(counts), offsets_of(counts)
    x, dy = normal(g, S, K, std=x_std, dtype=F16), normal(g, S, N, std=dy_std, dtype=F16)
    a, b = normal(g, n, r, K, std=a_std, dtype=F16), normal(g, n, N, r, std=b_std, dtype=F16)
    scale = (torch.rand(n, generator=g, device="cuda") + 0.5) * f
    _, u = B.situ_moe_lora(torch.zeros(S, N, device="cuda"), x, a, b, offsets=off, scale=scale, keep=True)
    _, da, db = B.situ_moe_lora_backward(dy, x, a, b, off, u, scale=scale)
    for e, (v, va, xe), (ue, ua, de) in gradients(dy, x, a, b, counts, scale):
        for got, p, pa, t, C, kept in ((da[e], v, va, xe, N, False), (db[e].T, ue, ua, de, K, True)):
            want = p.T @ t
            assert want.abs().max() < 3e4 if len(p) else True     # the results themselves are f16's
            within(got, want, far_bar(want, p, pa, t, C, kept))
    again = B.situ_moe_lora_backward(dy, x, a, b, off, u, scale=scale)
    assert torch.equal(again[1], da) and torch.equal(again[2], db)


def test_f16_gradients_of_rows_of_every_size():
    # in one adapter rows that the kept terms hold, rows beyond f16, tiny rows and zeros; NaN next door stays there
    g = gen(3)
    counts, K, N, r = [130, 70], 264, 136, 24
    S, off = sum(counts), offsets_of(counts)
    x = normal(g, S, K) * torch.tensor([1.0, 3e4, 1e-5, 0.0, 100.0], device="cuda")[torch.arange(S, device="cuda") % 5][:, None]
    x, dy = x.clamp(-6e4, 6e4).to(F16), normal(g, S, N, std=1e-5, dtype=F16)
    a, b = normal(g, 2, r, K, dtype=F16), normal(g, 2, N, r, std=1e-3, dtype=F16)
    scale = torch.tensor([1.0, -0.5], device="cuda")
    x[135], a[1, 3] = float("inf"), float("nan")
    _, u = B.situ_moe_lora(None, x, a, b, offsets=off, scale=scale, keep=True)
    _, da, db = B.situ_moe_lora_backward(dy, x, a, b, off, u, scale=scale)
    _, (v, va, xe), (ue, ua, de) = next(gradients(dy, x, a, b, counts, scale))
    for got, p, pa, t, C, kept in ((da[0], v, va, xe, N, False), (db[0].T, ue, ua, de, K, True)):
        want = p.T @ t
        within(got, want, far_bar(want, p, pa, t, C, kept))
    assert torch.isnan(db[1, :, 3]).all() and torch.isfinite(db[0]).all() and torch.isfinite(da[0]).all()
