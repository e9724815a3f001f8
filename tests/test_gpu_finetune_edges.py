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
        yield (e, (f * (de @ be), f.abs() * (de.abs() @ be.abs()), xe),
               (f * (xe @ ae.T), f.abs() * (xe.abs() @ ae.abs().T), de))


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
# --------------------------------------------------------------------------
# gated activation near zero, beside large caps and far below it
# --------------------------------------------------------------------------

def factors(x, cap):
    """cap tanh(x / cap) and its derivative in 64 bits; x and 1 without a cap."""
    if cap <= 0:
        return x, torch.ones_like(x)
    y = x / cap
    s = torch.exp(-2 * y.abs())
    return cap * torch.tanh(y), 4 * s / (1 + s) ** 2


# Relative errors.  A factor cap tanh(x / cap): where |x / cap| >= 2^-7.5 the exponential is off by 2^-22 and the
# difference 1 - e^(-2 x / cap) is at least 2^-6.5, so off by 2^-15.5; below, by the 2^-16.5 that tanh(y)/y is short of
# 1.  A sigmoid: 2^-22 and 2^-23.4 of its argument's magnitude, below 2^-16.9 for |g| <= 80.  Two factors, a sigmoid and
# roundings: below 2^-14.  A derivative is off by 2^-15 where x counts as 2^-7.5: a fifth more.
NEAR = 2.0 ** -14
CAPS = [0.5, 1.7, 30.0, 2.0 ** 12, 3e6, 1e9, 1e30, 0.0]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("b", CAPS)
@pytest.mark.parametrize("bl", [0.7, 1e8, -1.0])
@pytest.mark.parametrize("far", [False, True])
def test_situ_is_rounded_once(dtype, b, bl, far):
    # magnitudes from 2^-20 to 4, or to 80; in blocks of mixed and of like size (8 bits keep a block's largest)
    g = gen(7)
    S, I = 96, 64
    size = torch.rand(S, 2 * I, generator=g, device="cuda") * (27.3 if far else 22) - 20
    size[::3] = size[::3, :1]
    size = size.clamp(max=6.32 if far else 2.0)
    x = (torch.exp2(size) * (torch.randint(0, 2, size.shape, generator=g, device="cuda") * 2 - 1)).to(dtype)
    p0, p1 = torch.tensor([b], device="cuda"), torch.tensor([bl], device="cuda")
    h, q, s = B.situ_moe_gated(x, p0, p1, save=True)
    tiny = TINY[dtype] + 2.0 ** -118           # a sigmoid below 2^-126 is zero

    def parts(x):
        gg, u = x.double().chunk(2, 1)
        (t, dt), (up, dup) = factors(gg, p0.item()), factors(u, p1.item())
        sg, cg = torch.sigmoid(gg), torch.sigmoid(-gg)
        return t * sg, dt * sg, t * sg * cg, up, dup

    gate, _, _, up, _ = parts(x)
    want = gate * up
    within(h, want, (H[dtype] + NEAR) * want.abs() + tiny)
    assert torch.equal(B.situ_moe_gated(x, p0, p1), h)
    back = B.situ_moe_restore_mxfp8(q.reshape(2 * S, I), s.reshape(2 * S, -1), F32).reshape(S, 2 * I)
    dh = normal(g, S, I, dtype=dtype)
    dx, h2 = B.situ_moe_gated_backward(dh, q, s, p0, p1, want_h=True)
    gate, d0, d1, up, dup = parts(back)
    within(h2, gate * up, (H[dtype] + NEAR) * (gate * up).abs() + tiny)
    d = dh.double()
    want = d * (d0 + d1) * up
    # the slope's two terms may cancel: their own errors, not their sum's
    within(dx[:, :I], want, H[dtype] * want.abs() + 1.2 * NEAR * (d * up).abs() * (d0 + d1.abs()) + tiny)
    want = d * gate * dup
    within(dx[:, I:], want, (H[dtype] + 1.2 * NEAR) * want.abs() + tiny)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", [B.SITU_ACT_FN_SITU, B.SITU_ACT_FN_SWIGLU_BIAS])
def test_gated_values_do_not_depend_on_their_neighbours(dtype, act):
    # gates below -25 beside ordinary and beside large ones, each as its limit has it
    I = 64
    g = torch.linspace(-80, -20, I, device="cuda")
    x = torch.stack([torch.cat((g, torch.full((I,), 1.5, device="cuda")))] * 2).to(dtype)
    x[1, ::16] = 3e4                             # another form of the arithmetic for these lanes' columns
    for p in ((0.7, 1.9), (0.0, 0.0)) if act == B.SITU_ACT_FN_SITU else ((1.0, 0.5),):
        p0, p1 = torch.tensor([p[0]], device="cuda"), torch.tensor([p[1]], device="cuda")
        h = B.situ_moe_gated(x, p0, p1, activation=act)
        gg = x[:, :I].double()
        if act == B.SITU_ACT_FN_SITU:
            want = factors(gg, p[0])[0] * torch.sigmoid(gg) * factors(x[:, I:].double(), p[1])[0]
        else:
            want = gg * torch.sigmoid(gg) * (x[:, I:].double() + p[1])
        same = torch.arange(I, device="cuda") % 16 != 0
        within(h[:, same], want[:, same], (H[dtype] + NEAR) * want[:, same].abs() + TINY[dtype])
        assert ((h[0, same].double() - h[1, same].double()).abs() <= (2 * H[dtype] + 2 * NEAR) * want[0, same].abs()
                + TINY[dtype]).all()
# --------------------------------------------------------------------------
# router: masked rows whose weights are NaN
# --------------------------------------------------------------------------

@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [24, 200, 1500])
def test_masked_tokens_of_any_logits_get_no_gradient(renorm, E):
    T, k = 40, 3
    g = gen(E)
    logits, mask = torch.randn(T, E, generator=g, device="cuda"), torch.ones(T, dtype=torch.bool, device="cuda")
    rows = [3, 11, 17, 39]
    mask[rows] = False
    dw = torch.randn(T, k, generator=g, device="cuda") * mask[:, None]       # the loss does not see them
    want = logits.clone().requires_grad_()
    _, w, _, loss = B.balanced_route(want, k, renormalize=renorm, mask=mask)
    torch.autograd.backward((w, loss), (dw, torch.ones_like(loss)))
    bad = logits.clone()
    bad[3], bad[11], bad[17], bad[39, 5] = -float("inf"), float("inf"), float("nan"), float("nan")
    leaf = bad.requires_grad_()
    _, w, _, loss = B.balanced_route(leaf, k, renormalize=renorm, mask=mask)
    torch.autograd.backward((w, loss), (dw, torch.ones_like(loss)))
    assert (leaf.grad[rows] == 0).all() and torch.equal(leaf.grad[mask], want.grad[mask])
    assert torch.isfinite(leaf.grad).all()


# --------------------------------------------------------------------------
# adapters beside an fp32 projection
# --------------------------------------------------------------------------

@pytest.mark.parametrize("size", [1e-30, 1e-9, 1.0, 1e7])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_fp32_gradients_beside_16_bit_operands(dtype, size):
    g = gen(11)
    counts, K, N, r = [60, 0, 41], 136, 72, 8
    S, n, off = sum(counts), len(counts), offsets_of(counts)
    inv = 1.0 / size                                    # brings the results back into f16's range where it can
    x = normal(g, S, K, std=min(inv, 3e3), dtype=dtype)
    a, b = normal(g, n, r, K, std=0.1, dtype=dtype), normal(g, n, N, r, std=min(inv, 1e3), dtype=dtype)
    leaves = [t.requires_grad_() for t in (torch.randn(S, N, generator=g, device="cuda"), x, a, b)]
    dy = torch.randn(S, N, generator=g, device="cuda") * size
    B.lora_linear(*leaves, off).backward(dy)
    assert torch.equal(leaves[0].grad, dy)
    x, a, b = (t.detach() for t in leaves[1:])
    most = dy.abs().max().double() if dtype is F16 else 0.0
    # dy rounded to the operands' type, in f16 under a power of two (half a subnormal's step, 2^-25, beside 2^14); what
    # the two terms leave (bf16 2^-17, f16 2^-22); the rest as above
    terms16 = 2.0 ** -17 if dtype is BF16 else 2.0 ** -22
    for e, (v, va, xe), (ue, ua, de) in gradients(dy, x, a, b, counts, torch.ones(n, device="cuda")):
        if not counts[e]:
            assert (leaves[2].grad[e] == 0).all() and (leaves[3].grad[e] == 0).all()
            continue
        L = counts[e]
        want, terms = v.T @ xe, v.abs().T @ xe.abs()
        within(leaves[2].grad[e], want, 1.1 * H[dtype] * want.abs() + (H[dtype] + (2 * L + 2 * N + 80) * U) * (va.T @ xe.abs())
               + terms16 * terms + 2.0 ** -39 * (most * b[e].double().abs().sum(0) + v.abs().max())[:, None] * xe.abs().sum(0)
               + TINY[dtype] / 2)
        want, terms = de.T @ ue, de.abs().T @ ue.abs()
        within(leaves[3].grad[e], want, 1.1 * H[dtype] * want.abs() + (H[dtype] + terms16 + 2 * L * U) * terms
               + (2 * K + 80) * U * (de.abs().T @ ua) + 2.0 ** -39 * most * ue.abs().sum(0)
               + (2.0 ** -25 + 2.0 ** -39 * ue.abs().max()) * de.abs().sum(0)[:, None] + TINY[dtype] / 2)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_dy_scale(dtype):
    # a power of two changes no bit beside dy that has it
    g = gen(12)
    counts, K, N, r = [300, 41], 136, 264, 16
    S, off = sum(counts), offsets_of(counts)
    x, dy = normal(g, S, K, dtype=dtype), normal(g, S, N, dtype=dtype)
    a, b = normal(g, 2, r, K, std=0.1, dtype=dtype), normal(g, 2, N, r, std=0.3, dtype=dtype)
    scale = torch.tensor([0.7, -1.3], device="cuda")
    _, u = B.situ_moe_lora(None, x, a, b, offsets=off, scale=scale, keep=True)
    for f in (0.125, 4.0, -1.0):
        t = torch.tensor([f], device="cuda")
        for p, q in zip(B.situ_moe_lora_backward(dy, x, a, b, off, u, scale=scale, dy_scale=t),
                        B.situ_moe_lora_backward(dy * f, x, a, b, off, u, scale=scale)):
            assert torch.equal(p, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p = B.situ_moe_lora_backward(dy, x, a, b, off, u, scale=scale, dy_scale=t, stream=s)
    s.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(p, B.situ_moe_lora_backward(dy * f, x, a, b, off, u, scale=scale)))
    for bad in (torch.ones(2, device="cuda"), torch.ones(1), torch.ones(1, device="cuda", dtype=dtype)):
        with pytest.raises(ValueError, match="dy_scale"):
            B.situ_moe_lora_backward(dy, x, a, b, off, u, dy_scale=bad)


@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_adapters_beyond_those_that_are_sorted(order):
    # more adapters than any sort here takes: tiles of as many adapters as rows
    g = gen(21)
    S, K, N, r, n = 3001, 72, 136, 8, 5000
    x, a, b = normal(g, S, K), normal(g, n, r, K, std=0.1), normal(g, n, N, r, std=0.3)
    base, ids = normal(g, S, N), torch.randint(-3, n + 3, (S,), generator=g, device="cuda").int()
    if order == "runs":
        ids = ids.sort().values
    y = B.situ_moe_lora(base, x, a, b, ids=ids)
    none = (ids < 0) | (ids >= n)
    e = ids.clamp(0, n - 1).long()
    xd, ad, bd = x.double(), a[e].double(), b[e].double()
    u = torch.einsum("sk,srk->sr", xd, ad)
    want = torch.einsum("sr,snr->sn", u, bd) * ~none[:, None] + base.double()
    both = torch.einsum("sr,snr->sn", torch.einsum("sk,srk->sr", xd.abs(), ad.abs()), bd.abs())
    second = torch.einsum("sr,snr->sn", u.abs(), bd.abs())
    within(y, want, H[BF16] * want.abs() + (2 * K + 40) * U * both + (H[BF16] + (6 * r + 8) * U) * second + TINY[BF16])
    assert torch.equal(y[none], base[none])


# --------------------------------------------------------------------------
# captures
# --------------------------------------------------------------------------

def test_a_capture_beside_nodes_kept_from_a_side_stream():
    # the usual recipe: a warm-up on a side stream, a wrapper that keeps the leaves' nodes, and a graph on its own stream
    g = gen(31)
    S, K, N, r = 300, 72, 64, 8
    x, dy = normal(g, S, K), normal(g, S, N)
    a, b = normal(g, 2, r, K).requires_grad_(), normal(g, 2, N, r).requires_grad_()
    off, base = offsets_of([100, 200]), torch.zeros(S, N, dtype=BF16, device="cuda")
    B.lora_linear(base, x, a, b, off).backward(dy)
    want, a.grad, b.grad = (a.grad.clone(), b.grad.clone()), None, None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kept = [t.expand_as(t).grad_fn.next_functions[0][0] for t in (a, b)]
        for _ in range(2):
            B.lora_linear(base, x, a, b, off).backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    a.grad = b.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.lora_linear(base, x, a, b, off).backward(dy)
    x.mul_(2.0)                                  # a power of two, through every rounding
    for _ in range(2):
        graph.replay()
    assert torch.equal(a.grad, 2 * want[0]) and torch.equal(b.grad, 2 * want[1]) and len(kept) == 2


def test_a_captured_step_of_f16_adapters_beside_an_fp32_base():
    g = gen(33)
    S, K, N, r = 200, 72, 64, 8
    x, base, dy = normal(g, S, K, dtype=F16), normal(g, S, N, dtype=F32), normal(g, S, N, std=1e-9, dtype=F32)
    a, b = normal(g, 2, r, K, dtype=F16).requires_grad_(), normal(g, 2, N, r, std=100.0, dtype=F16).requires_grad_()
    off = offsets_of([120, 80])

    def run():
        return torch.autograd.grad(B.lora_linear(base, x, a, b, off), (a, b), dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for size in (1e-6, 1e3, 0.0):
        dy.copy_(normal(g, S, N, std=size, dtype=F32))
        graph.replay()
        want = run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # dB has a deviation of size 72^0.5 120^0.5 = 93 size: at 1e3 many of its elements are beyond f16
        true = torch.stack([dy[q].double().T @ (x[q].double() @ a[e].double().T) for e, q in ((0, slice(0, 120)), (1, slice(120, 200)))])
        assert torch.isfinite(got[1][true.abs() < 6e4]).all() and (got[1].abs().max() > 0) == (size > 0)
