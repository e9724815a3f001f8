"""The fine-tuning operators on the GPU against plain implementations in 64
bits: the router's balance loss and gradient, the gated activation with its
input in 8 bits and its backward pass, low-rank adapters and their gradients.

The bars count roundings.  H: half an ulp of a 16-bit type, relative.  An fp32
operation is off by U = 2^-24 relative.  The tensor cores truncate when they
add: 2 U of the sum of the terms' magnitudes per term at most.
"""
import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
H = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -133, F16: 2.0 ** -24, F32: 2.0 ** -149}    # the least magnitude above zero
U = 2.0 ** -24
SITU, SWIGLU = B.SITU_ACT_FN_SITU, B.SITU_ACT_FN_SWIGLU_BIAS


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()
    yield
    assert B.situ_moe_gemm_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offsets_of(counts):
    return torch.tensor([0] + list(counts), device="cuda").cumsum(0).int()


def within(got, want, bar):
    got = got.double()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - bar
    assert (off <= 0).all(), (off.max().item(), (off > 0).sum().item())


# --------------------------------------------------------------------------
# router
# --------------------------------------------------------------------------

def router_case(T, E, k, seed=0, spread=1.5):
    g = gen(seed + 31 * T + E)
    logits = torch.randn(T, E, generator=g, device="cuda") * spread
    dw = torch.randn(T, k, generator=g, device="cuda") * 0.1
    return logits, dw


def router_ref(logits, ids, mask, coef, dloss, dw, renorm):
    """(loss, counts, dlogits, bar of dlogits per unit of a probability's relative error) in 64 bits."""
    T, E = logits.shape
    k = ids.shape[1]
    l = logits.double()
    p = torch.softmax(l, 1)
    m = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    n = int(m.sum())
    live = ids[m].long()
    live = live[(live >= 0) & (live < E)]
    counts = torch.bincount(live, minlength=E)
    f = counts.double() / max(1, n * k)
    loss = coef * E * (f * p[m].sum(0) / max(1, n)).sum()
    c = coef * E / max(1, n) * dloss
    dot = (p * f).sum(1, keepdim=True)
    d = c * p * (f - dot) * m[:, None]
    bar = abs(c) * p * (f + dot) * m[:, None]
    if dw is not None:
        ok = (ids >= 0) & (ids < E)
        at = ids.long().clamp(0, E - 1)
        w = torch.where(ok, torch.softmax(torch.where(ok, l.gather(1, at), -torch.inf), 1) if renorm else p.gather(1, at), 0.0)
        wd = w * dw.double()
        s, a = wd.sum(1, keepdim=True), wd.abs().sum(1, keepdim=True)
        if renorm:
            d = d.scatter_add(1, at, wd - w * s)
            bar = bar.scatter_add(1, at, wd.abs() + w * a)
        else:
            d = d.scatter_add(1, at, wd) - p * s
            bar = bar.scatter_add(1, at, wd.abs()) + p * a
    return loss, counts, d, bar


# A probability's relative error: |l - max| U for the difference and twice
# |l - max| log2(e) ln(2) U for its product with a rounded constant (3 D U), 4 U
# of the exponential, 64 U of the row's sum (32 additions in a lane, up to 8
# across, and the terms' own), 3 U of reciprocal and products.  Twice that for a
# term with a sum of such over a row, and as much again for a weight.
def p_error(logits):
    spread = (logits.amax(1, keepdim=True) - logits).clamp(max=100).amax().item()
    return (3 * spread + 4 + 64 + 3) * U


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (32, 8, 8), (3, 3, 2), (70, 64, 4), (257, 65, 5), (300, 128, 16),
                                   (1000, 130, 6), (513, 256, 8), (95, 385, 3), (2000, 512, 2), (129, 770, 16),
                                   (4099, 896, 16), (300, 1024, 10), (77, 1025, 3), (64, 2048, 16), (41, 2052, 7),
                                   (33, 4096, 16), (9, 4095, 16), (40001, 130, 6), (40000, 256, 8), (90000, 37, 3)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("masked", [False, True])
def test_router(T, E, k, renorm, masked):
    logits, dw = router_case(T, E, k)
    mask = torch.rand(T, generator=gen(T), device="cuda") < 0.6 if masked else None
    ids, w = B.situ_moe_route_topk(logits, k, renorm)
    coef, dloss = 0.37, torch.tensor(1.7, device="cuda")
    loss, counts, tokens, stats = B.situ_moe_balance_loss(logits, ids, mask=mask, coef=coef)
    d = B.situ_moe_router_backward(logits, ids, counts, tokens, stats, dloss=dloss, coef=coef, mask=mask, topk_weights=w,
                                   dweights=dw, renormalize=renorm)
    rl, rc, rd, bar = router_ref(logits, ids, mask, coef, float(dloss), dw, renorm)
    assert torch.equal(counts.long(), rc) and int(tokens) == (T if mask is None else int(mask.sum()))
    e = p_error(logits)
    assert abs(loss.item() - rl.item()) <= (e + 512 * U) * abs(rl.item())     # up to 512 rows in a lane's sum
    within(d, rd, 4 * e * bar + 1e-30)
    # the parts one by one, whatever the other would have read
    only = B.situ_moe_router_backward(logits, ids, counts, tokens, stats, dloss=dloss, coef=coef, mask=mask)
    _, _, r1, b1 = router_ref(logits, ids, mask, coef, float(dloss), None, renorm)
    within(only, r1, 4 * e * b1 + 1e-30)
    only = B.situ_moe_router_backward(logits, ids, None, None, stats, topk_weights=w, dweights=dw, renormalize=renorm)
    _, _, r2, b2 = router_ref(logits, ids, mask, 0.0, 0.0, dw, renorm)
    within(only, r2, 4 * e * b2 + 1e-30)


def test_router_gradient_by_differences():
    T, E, k = 12, 40, 3
    logits, dw = router_case(T, E, k, seed=5)
    ids, w = B.situ_moe_route_topk(logits, k, True)
    loss, counts, tokens, stats = B.situ_moe_balance_loss(logits, ids, coef=2.0)
    d = B.situ_moe_router_backward(logits, ids, counts, tokens, stats, dloss=torch.ones((), device="cuda"), coef=2.0)
    step = 2.0 ** -5
    p, f = torch.softmax(logits.double(), 1), (counts.double() / (T * k)).max().item()
    for t, e in ((0, 3), (5, 17), (11, 39)):
        at = []
        for s in (step, -step):
            l = logits.clone()
            l[t, e] += s
            at.append(B.situ_moe_balance_loss(l, ids, coef=2.0)[0].item())   # the IDs held: f_e are constants
        # central differences: step^2 / 6 of the third derivative, which is below p for the logit's own probability and
        # below 6 p in all for the others', and both losses' errors over 2 step
        bar = 2 * E / T * 7 * 1.1 * p[t, e].item() * f * step ** 2 / 6 + 2 * (p_error(logits) + 8 * U) * at[0] / (2 * step)
        assert abs((at[0] - at[1]) / (2 * step) - d[t, e].item()) <= bar


def test_router_edges():
    T, E, k = 50, 100, 4
    logits, dw = router_case(T, E, k)
    ids, w = B.situ_moe_route_topk(logits, k, True)
    want = B.situ_moe_balance_loss(logits, ids, coef=1.0)
    # even routing: exactly coef
    even = torch.zeros(8, 8, device="cuda")
    loss, counts, _, _ = B.situ_moe_balance_loss(even, torch.arange(8, device="cuda", dtype=torch.int32)[:, None], coef=0.5)
    assert abs(loss.item() - 0.5) <= 0.5 * 4 * U and (counts == 1).all()
    # strided rows, off 16 bytes too
    for pad, skip in ((4, 0), (3, 0), (5, 1)):
        wide = torch.full((T, E + pad), float("nan"), device="cuda")
        view = wide[:, skip:skip + E]
        view.copy_(logits)
        got = B.situ_moe_balance_loss(view, ids, coef=1.0)
        assert torch.equal(got[1], want[1]) and abs(got[0] - want[0]) <= 8 * U * want[0]
        out = torch.full((T, E + 8), 7.0, device="cuda")
        a = B.situ_moe_router_backward(view, ids, *want[1:], dloss=torch.ones((), device="cuda"), out=out[:, :E])
        b = B.situ_moe_router_backward(logits, ids, *want[1:], dloss=torch.ones((), device="cuda"))
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-9) and (out[:, E:] == 7).all()
    # masked rows may hold anything, and get no gradient
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[[3, 10, 49]] = False
    bad = logits.clone()
    bad[3], bad[10], bad[49] = float("nan"), float("inf"), -float("inf")
    base = B.situ_moe_balance_loss(logits, ids, mask=mask, coef=1.0)
    got = B.situ_moe_balance_loss(bad, ids, mask=mask, coef=1.0)
    assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1]) and int(got[2]) == T - 3
    one = torch.ones((), device="cuda")
    d = B.situ_moe_router_backward(bad, ids, *got[1:], dloss=one, mask=mask, topk_weights=w,
                                   dweights=torch.where(mask[:, None], dw, 0.0))
    assert torch.isfinite(d).all() and (d[~mask] == 0).all()
    ref = B.situ_moe_router_backward(logits, ids, *base[1:], dloss=one, mask=mask, topk_weights=w,
                                     dweights=torch.where(mask[:, None], dw, 0.0))
    assert torch.equal(d[mask], ref[mask])
    # experts masked by -inf or the type's lowest: no probability, no gradient
    for low in (-float("inf"), torch.finfo(F32).min):
        l = logits.clone()
        l[:, 60:] = low
        i2, w2 = B.situ_moe_route_topk(l, k, False)
        loss, counts, tokens, stats = B.situ_moe_balance_loss(l, i2)
        d = B.situ_moe_router_backward(l, i2, counts, tokens, stats, dloss=one, topk_weights=w2, dweights=dw, renormalize=False)
        assert torch.isfinite(d).all() and (d[:, 60:] == 0).all() and (counts[60:] == 0).all() and torch.isfinite(loss)
    # a row of -inf has no probabilities
    l = logits.clone()
    l[7] = -float("inf")
    loss, counts, tokens, stats = B.situ_moe_balance_loss(l, ids)
    d = B.situ_moe_router_backward(l, ids, counts, tokens, stats, dloss=one)
    assert torch.isfinite(loss) and (d[7] == 0).all()
    # a NaN shows
    l[7, 3] = float("nan")
    loss, counts, tokens, stats = B.situ_moe_balance_loss(l, ids)
    assert torch.isnan(loss) and torch.isnan(B.situ_moe_router_backward(l, ids, counts, tokens, stats, dloss=one)[7]).all()
    # no token, or none left
    loss, counts, tokens, _ = B.situ_moe_balance_loss(logits[:0], ids[:0])
    assert loss.item() == 0 and (counts == 0).all() and int(tokens) == 0
    loss, counts, tokens, stats = B.situ_moe_balance_loss(logits, ids, mask=torch.zeros(T, dtype=torch.uint8, device="cuda"))
    assert loss.item() == 0 and (counts == 0).all() and int(tokens) == 0
    assert (B.situ_moe_router_backward(logits, ids, counts, tokens, stats, dloss=one) == 0).all()


@pytest.mark.parametrize("E", [8, 100, 500, 3000])
def test_router_ids_outside_and_named_twice(E):
    T, k = 90, 8
    logits, dw = router_case(T, E, k)
    ids = torch.randint(-2, E + 2, (T, k), generator=gen(E), device="cuda").int()
    ids[::3, 1] = ids[::3, 0]
    ids[::3, 5] = ids[::3, 0]
    ids[1::9] = ids[1::9, :1]
    ok = (ids >= 0) & (ids < E)
    w = torch.softmax(logits, 1).gather(1, ids.long().clamp(0, E - 1)) * ok
    loss, counts, tokens, stats = B.situ_moe_balance_loss(logits, ids, coef=1.0)
    rl, rc, rd, bar = router_ref(logits, ids, None, 1.0, 1.0, dw, False)
    assert torch.equal(counts.long(), rc)
    first = None
    for _ in range(3):
        d = B.situ_moe_router_backward(logits, ids, counts, tokens, stats, dloss=torch.ones((), device="cuda"), coef=1.0,
                                       topk_weights=w, dweights=dw, renormalize=False)
        within(d, rd, 4 * p_error(logits) * bar + 1e-30)
        first = d if first is None else first
        assert torch.equal(d, first)


def test_router_long_rows_of_tokens():
    # many rows per CTA, and the same bits every time
    T, E, k = 70001, 60, 4
    logits, _ = router_case(T, E, k)
    ids, _ = B.situ_moe_route_topk(logits, k)
    loss, counts, tokens, _ = B.situ_moe_balance_loss(logits, ids)
    rl, rc, _, _ = router_ref(logits, ids, None, 1.0, 1.0, None, True)
    assert torch.equal(counts.long(), rc) and int(tokens) == T
    assert abs(loss.item() - rl.item()) <= (p_error(logits) + 512 * U) * rl.item()
    for _ in range(3):
        assert torch.equal(B.situ_moe_balance_loss(logits, ids)[0], loss)


def test_router_many_rows_a_group():
    # column sums taken out of the registers several times
    T, E, k = 1_500_001, 20, 2
    logits, _ = router_case(T, E, k)
    ids, _ = B.situ_moe_route_topk(logits, k)
    loss, counts, tokens, _ = B.situ_moe_balance_loss(logits, ids)
    rl, rc, _, _ = router_ref(logits, ids, None, 1.0, 1.0, None, True)
    assert torch.equal(counts.long(), rc) and int(tokens) == T
    assert abs(loss.item() - rl.item()) <= (p_error(logits) + (256 + 32 + 2 * 16) * U) * rl.item()


def test_balanced_route_gradients():
    T, E, k = 60, 24, 3
    logits, dw = router_case(T, E, k)
    leaf = logits.clone().requires_grad_()
    ids, w, counts, loss = B.balanced_route(leaf, k, coef=0.3)
    ((w * dw).sum() + 2.0 * loss).backward()
    _, rc, rd, bar = router_ref(logits, ids, None, 0.3, 2.0, dw, True)
    within(leaf.grad, rd, 4 * p_error(logits) * bar + 1e-30)
    assert torch.equal(counts.long(), rc) and not ids.requires_grad
    for f in (lambda w, loss: (w * dw).sum(), lambda w, loss: loss):         # one of the two alone
        leaf.grad = None
        ids, w, counts, loss = B.balanced_route(leaf, k, coef=0.3)
        f(w, loss).backward()
        assert torch.isfinite(leaf.grad).all()


# --------------------------------------------------------------------------
# 8 bits
# --------------------------------------------------------------------------

def plain_save(x):
    """The rule on the CPU, in fp32 (every step exact but the last): (codes, bytes)."""
    x = x.cpu().float()
    S, K = x.shape
    b = torch.nn.functional.pad(x, (0, -K % 32)).reshape(S, -1, 32)
    amax = b.abs().amax(-1)
    m, p = torch.frexp(amax)
    e = torch.where(amax > 0, torch.where(m > 0.875, p - 8, p - 9), -127).clamp(-127, 127)
    q = (b.double() * torch.ldexp(torch.ones((), dtype=F64), -e.double())[..., None]).float()
    q = q.to(torch.float8_e4m3fn).view(torch.uint8)
    lost = ~torch.isfinite(b).all(-1)
    q[lost], byte = 0x7F, torch.where(lost, 255, e + 127).to(torch.uint8)
    return q.reshape(S, -1)[:, :K].contiguous(), byte


def plain_restore(q, byte):
    f = torch.where(byte == 255, torch.nan, torch.ldexp(torch.ones((), dtype=F64), byte.double() - 127))
    return q.view(torch.float8_e4m3fn).double() * f.repeat_interleave(32, -1)[:, : q.shape[1]]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("S,K", [(1, 8), (1, 32), (3, 40), (17, 264), (130, 1000), (65, 2072), (9, 4096), (2, 16392)])
def test_save_and_restore(dtype, S, K):
    g = gen(S + K)
    x = (torch.randn(S, K, generator=g, device="cuda") * torch.exp2(torch.rand(S, 1, generator=g, device="cuda") * 24 - 14))
    x = x.to(dtype)
    x[:, ::7] = 0
    x[:, 1::11] = -0.0
    q, s = B.situ_moe_save_mxfp8(x)
    rq, rs = plain_save(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)
    if dtype is BF16 and K % 32 == 0:
        for a, b in zip((q, s), B.situ_moe_quant_mxfp8(x)):
            assert torch.equal(a, b)
    want = plain_restore(rq, rs)
    for t in (BF16, F16, F32):
        got = B.situ_moe_restore_mxfp8(q, s, t)
        # exact, up to the type's range and its subnormals
        assert torch.equal(got.cpu(), want.clamp(-torch.finfo(t).max, torch.finfo(t).max).to(t))
    # strides, given results, a copy where rows are off 16 bytes
    wide = torch.zeros(S, K + 16, dtype=dtype, device="cuda")
    for skip in (0, 8, 3):
        wide[:, skip:skip + K] = x
        a, b = B.situ_moe_save_mxfp8(wide[:, skip:skip + K])
        assert torch.equal(a, q) and torch.equal(b, s)
    back = torch.full((S, K + 8), 5.0, dtype=dtype, device="cuda")
    B.situ_moe_restore_mxfp8(q, s, dtype, out=back[:, :K])
    assert torch.equal(back[:, :K], B.situ_moe_restore_mxfp8(q, s, dtype)) and (back[:, K:] == 5).all()
    B.situ_moe_save_mxfp8(x, out=(q.fill_(1), s.fill_(1)))
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_save_at_the_ends_of_the_range(dtype):
    top, fi = torch.finfo(dtype).max, torch.finfo(dtype)
    x = torch.zeros(8, 96, dtype=dtype, device="cuda")
    x[0], x[1, ::2], x[2] = top, -top, fi.tiny
    x[3] = torch.arange(1, 97, device="cuda").to(dtype) * TINY[dtype]
    x[4, 3], x[5, 40], x[6, 95] = float("inf"), -float("inf"), float("nan")
    x[4, 50] = x[5, 2] = x[6, 0] = 1.5
    q, s = B.situ_moe_save_mxfp8(x)
    rq, rs = plain_save(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)
    got = B.situ_moe_restore_mxfp8(q, s, dtype)
    lost = (~torch.isfinite(x.cpu().reshape(8, 3, 32)).all(-1)).repeat_interleave(32, -1)
    assert torch.equal(torch.isnan(got.cpu()), lost)
    assert torch.isfinite(got[:4]).all() and (got[0] == top).all()
    want = plain_restore(rq, rs).clamp(-top, top).to(dtype)
    assert torch.equal(got.cpu()[~lost], want[~lost])


# --------------------------------------------------------------------------
# gated activation
# --------------------------------------------------------------------------

def expert_rows(offsets, S):
    row = torch.arange(S, device="cuda")
    e = torch.searchsorted(offsets.long()[1:], row, right=True)
    return e.clamp(max=offsets.numel() - 2), (row >= offsets[0]) & (e < offsets.numel() - 1)


def gated_ref(x, p0, p1, act):
    """(h, dh/dg, dh/du, and bounds A, B of the two factors) in 64 bits; p0, p1 as columns."""
    g, u = x.double().chunk(2, 1)
    p0, p1 = p0.double(), p1.double()
    if act == SITU:
        sg = torch.sigmoid(g)
        c0, c1 = torch.where(p0 > 0, p0, 1.0), torch.where(p1 > 0, p1, 1.0)
        t, dt = torch.where(p0 > 0, c0 * torch.tanh(g / c0), g), torch.where(p0 > 0, torch.cosh(g / c0) ** -2, 1.0)
        up, du = torch.where(p1 > 0, c1 * torch.tanh(u / c1), u), torch.where(p1 > 0, torch.cosh(u / c1) ** -2, 1.0)
        gate, dgate = t * sg, dt * sg + t * sg * (1 - sg)
        A, Bu = torch.where(p0 > 0, c0.expand_as(g), g.abs()), torch.where(p1 > 0, c1.expand_as(u), u.abs())
    else:
        sg = torch.sigmoid(p0 * g)
        gate, dgate = g * sg, sg + p0 * g * sg * (1 - sg)
        up, du = u + p1, torch.ones_like(u)
        A, Bu = g.abs(), u.abs() + p1.abs()
    return gate * up, dgate * up, gate * du, A, Bu


# The activation in fp32.  An exponential's argument is k x with k and the
# product rounded, its magnitude clamped at 36.1 (25 log2 e; SWIGLU_BIAS 115.5):
# 2 |z| ln(2) U = 50 U (160 U), and 4 U of the exponential: below 2^-18 (2^-16.6)
# relative.  tanh and sigmoid are off by at most that (their derivatives by
# log E are below 1), a product of three factors with the reciprocal and six
# roundings by three times that and 10 U: below 2^-16 (2^-14.9) of the factors'
# bounds.  The derivatives have two more factors: twice that.
F_ERR = {SITU: 2.0 ** -16, SWIGLU: 2.0 ** -14.5}


def caps(g, E, act):
    p0 = torch.rand(E, generator=g, device="cuda") * 2 + 0.3
    p1 = torch.rand(E, generator=g, device="cuda") * 2 + (0.3 if act == SITU else -1.0)
    if act == SITU:
        p0[2::5], p1[1::4] = 0.0, -1.0
    return p0, p1


COUNTS = [[1], [5], [300], [3, 0, 70, 1, 0, 129], [0, 0, 4], [17] * 40]


@pytest.mark.parametrize("act", [SITU, SWIGLU])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I", [8, 40, 200, 384, 2056])
def test_gated(act, dtype, counts, I):
    g = gen(I + len(counts))
    spare = 3 if len(counts) > 1 else 0
    S, E = sum(counts) + spare, len(counts)
    off = offsets_of(counts)
    p0, p1 = caps(g, E, act)
    x = normal(g, S, 2 * I, std=1.5, dtype=dtype)
    x[sum(counts):] = float("nan")                       # rows of no expert: not read
    e, held = expert_rows(off, S)
    h, q, s = B.situ_moe_gated(x, p0, p1, off, activation=act, save=True)
    assert torch.equal(B.situ_moe_gated(x, p0, p1, off, activation=act), h)
    live = torch.where(held[:, None], x, 0.0)
    ref, _, _, A, Bu = gated_ref(live, p0[e][:, None], p1[e][:, None], act)
    ref, A = ref * held[:, None], A * held[:, None]
    within(h, ref, H[dtype] * ref.abs() + (1 + H[dtype]) * F_ERR[act] * A * Bu + TINY[dtype] / 2)
    rq, rs = plain_save(live.reshape(2 * S, I))
    assert torch.equal(q.cpu().reshape(2 * S, I), rq) and torch.equal(s.cpu().reshape(2 * S, -1), rs)
    # backwards, at what was kept
    dh = normal(g, S, I, std=0.3, dtype=dtype)
    dx, h2 = B.situ_moe_gated_backward(dh, q, s, p0, p1, off, activation=act, want_h=True)
    back = plain_restore(rq, rs).reshape(S, 2 * I).cuda()
    ref, hg, hu, A, Bu = gated_ref(back, p0[e][:, None], p1[e][:, None], act)
    k, f = held[:, None], 2 * F_ERR[act]
    within(h2, ref * k, H[dtype] * ref.abs() + (1 + H[dtype]) * f * A * Bu + TINY[dtype] / 2)
    d = dh.double() * k
    slope = 1 + A * (1 if act == SITU else p0[e][:, None].double())
    within(dx[:, :I], d * hg, H[dtype] * (d * hg).abs() + d.abs() * f * (1 + H[dtype]) * slope * Bu + TINY[dtype] / 2)
    within(dx[:, I:], d * hu, H[dtype] * (d * hu).abs() + d.abs() * f * (1 + H[dtype]) * A + TINY[dtype] / 2)
    assert (dx[~held] == 0).all() and (h[~held] == 0).all() and (h2[~held] == 0).all()
    only, none = B.situ_moe_gated_backward(dh, q, s, p0, p1, off, activation=act)
    assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("act", [SITU, SWIGLU])
def test_gated_gradient_by_differences(act):
    # values that 8 bits hold exactly: the kept form is the input itself
    S, I = 6, 32
    g = gen(9)
    x = (torch.randint(-7, 8, (S, 2 * I), generator=g, device="cuda").float() / 4).to(F16)
    p0, p1 = torch.tensor([1.3], device="cuda"), torch.tensor([0.8], device="cuda")
    h, q, s = B.situ_moe_gated(x, p0, p1, activation=act, save=True)
    assert torch.equal(B.situ_moe_restore_mxfp8(q.reshape(2 * S, I), s.reshape(2 * S, -1), F16).reshape(S, 2 * I), x)
    dx, _ = B.situ_moe_gated_backward(torch.ones(S, I, dtype=F16, device="cuda"), q, s, p0, p1, activation=act)
    step = 2.0 ** -3                                     # exact in f16 beside multiples of 1/4
    for half in (0, 1):
        up, down = x.clone(), x.clone()
        up[:, half * I:(half + 1) * I] += step
        down[:, half * I:(half + 1) * I] -= step
        diff = (B.situ_moe_gated(up, p0, p1, activation=act).double() - B.situ_moe_gated(down, p0, p1, activation=act).double()) / (2 * step)
        # h's roundings over 2 step, and a third derivative below 8 (products of tanh and sigmoid, |x| < 2) times step^2 / 6
        bar = 2 * H[F16] * 4 / (2 * step) + 8 * step ** 2 / 6 + H[F16] * 4
        assert ((dx[:, half * I:(half + 1) * I].double() - diff).abs() <= bar).all()


@pytest.mark.parametrize("act", [SITU, SWIGLU])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gated_large_and_lost_values(act, dtype):
    I = 64
    big = torch.tensor([-1e4, -100.0, -30.0, -10.0, 0.0, 10.0, 30.0, 100.0, 1e4, 6e4], device="cuda")
    x = torch.cat((big.repeat_interleave(10)[:, None].expand(100, I), big.repeat(10)[:, None].expand(100, I)), 1).to(dtype)
    p0, p1 = torch.tensor([0.7], device="cuda"), torch.tensor([1.9], device="cuda")
    h, q, s = B.situ_moe_gated(x, p0, p1, activation=act, save=True)
    ref, _, _, A, Bu = gated_ref(x, p0[:, None], p1[:, None], act)
    top = torch.finfo(dtype).max
    ok = ref.abs() < top / 2
    assert ((h.double() - ref).abs() <= H[dtype] * ref.abs() + 2 * F_ERR[act] * A.clamp(max=1e5) * Bu + TINY[dtype])[ok].all()
    dx, _ = B.situ_moe_gated_backward(torch.ones(100, I, dtype=dtype, device="cuda"), q, s, p0, p1, activation=act)
    assert not torch.isnan(dx).any()
    # a NaN or an infinity shows where it was, and in the backward pass in its block of 32
    y = torch.zeros(4, 2 * I, dtype=dtype, device="cuda")
    y[0, 5], y[1, I + 40], y[2, 33] = float("nan"), float("nan"), float("inf")
    h, q, s = B.situ_moe_gated(y + 1, p0, p1, activation=act, save=True)
    assert torch.isnan(h[0, 5]) and torch.isnan(h[1, 40]) and torch.isnan(h).sum() <= 3 and torch.isfinite(h[3]).all()
    dx, _ = B.situ_moe_gated_backward(torch.ones(4, I, dtype=dtype, device="cuda"), q, s, p0, p1, activation=act)
    assert torch.isnan(dx[0, :32]).all() and torch.isnan(dx[1, 32:I]).all() and torch.isnan(dx[2, 32:I]).all()
    assert torch.isfinite(dx[0, 32:I]).all() and torch.isfinite(dx[3]).all()


def test_gated_strides_offsets_and_nothing():
    g = gen(4)
    counts, I = [20, 0, 31], 72
    off, S = offsets_of(counts), 51
    p0, p1 = caps(g, 3, SITU)
    x = normal(g, S, 2 * I)
    h, q, s = B.situ_moe_gated(x, p0, p1, off, save=True)
    wide = torch.zeros(S, 2 * I + 24, dtype=BF16, device="cuda")
    for skip in (0, 16, 5):
        wide[:, skip:skip + 2 * I] = x
        assert torch.equal(B.situ_moe_gated(wide[:, skip:skip + 2 * I], p0, p1, off), h)
    out = torch.full((S, I + 8), 3.0, dtype=BF16, device="cuda")
    B.situ_moe_gated(x, p0, p1, off, out=out[:, :I])
    assert torch.equal(out[:, :I], h) and (out[:, I:] == 3).all()
    dh = normal(g, S, I)
    dx, _ = B.situ_moe_gated_backward(dh, q, s, p0, p1, off)
    wide = torch.full((S, 2 * I + 8), 3.0, dtype=BF16, device="cuda")
    B.situ_moe_gated_backward(dh.t().contiguous().t(), q.view(torch.float8_e4m3fn), s, p0, p1, off, out=wide[:, :2 * I])
    assert torch.equal(wide[:, :2 * I], dx) and (wide[:, 2 * I:] == 3).all()
    # rows before the first expert's belong to none
    late = off + 7
    y = normal(g, 60, 2 * I)
    h = B.situ_moe_gated(y, p0, p1, late)
    assert (h[:7] == 0).all() and (h[58:] == 0).all()
    assert torch.equal(h[7:58], B.situ_moe_gated(y[7:58].contiguous(), p0, p1, off))
    h, q, s = B.situ_moe_gated(x[:0], p0, p1, torch.zeros(4, dtype=torch.int32, device="cuda"), save=True)
    assert h.shape == (0, I) and q.shape == (0, 2 * I)


# --------------------------------------------------------------------------
# adapters
# --------------------------------------------------------------------------

def lora_case(g, S, K, N, r, n, dtype, out_dtype):
    return dict(x=normal(g, S, K, dtype=dtype), a=normal(g, n, r, K, std=K ** -0.5, dtype=dtype),
                b=normal(g, n, N, r, std=r ** -0.5, dtype=dtype), base=normal(g, S, N, dtype=out_dtype),
                scale=torch.rand(n, generator=g, device="cuda") + 0.5)


def lora_ref(c, ids):
    """(y, |y's terms|: magnitudes through both products, magnitudes of u through the second, u) in 64 bits."""
    x, a, b, y = c["x"].double(), c["a"].double(), c["b"].double(), c["base"].double().clone()
    both, second, u = torch.zeros_like(y), torch.zeros_like(y), torch.zeros(len(ids), a.shape[1], dtype=F64, device="cuda")
    for e in range(a.shape[0]):
        rows = (ids == e).nonzero()[:, 0]
        if len(rows):
            f = c["scale"][e].double()
            u[rows] = f * (x[rows] @ a[e].T)
            y[rows] += u[rows] @ b[e].T
            both[rows] = f * ((x[rows].abs() @ a[e].abs().T) @ b[e].abs().T)
            second[rows] = u[rows].abs() @ b[e].abs().T
    return y, both, second, u


def lora_bar(y, both, second, K, r, dtype, out_dtype, rows):
    """Sums of K and r terms; u in 16 bits (by tiles), or with 22 bits or more;
    the splits' and the scale's roundings; the result's."""
    u16 = 0.0 if rows else H[dtype] if out_dtype is not F32 else 2.0 ** -21
    return H[out_dtype] * y.abs() + (2 * K + 40) * U * both + (u16 + (2 * r * 3 + 8) * U) * second + TINY[out_dtype]


@pytest.mark.parametrize("S,K,N,r,n", [(1, 8, 8, 8, 1), (1, 3584, 768, 16, 3), (5, 264, 1000, 24, 2), (33, 72, 136, 128, 40),
                                       (64, 128, 64, 40, 7), (65, 64, 128, 8, 2), (130, 200, 264, 16, 3), (300, 1032, 72, 32, 300),
                                       (700, 136, 1160, 48, 4), (1000, 520, 520, 64, 11), (257, 2048, 392, 128, 5),
                                       (2100, 64, 64, 104, 1), (3000, 136, 200, 24, 40), (2049, 520, 1032, 16, 700),
                                       (129, 64, 64, 128, 1), (200, 72, 136, 64, 2), (400, 64, 72, 128, 20),
                                       (60001, 64, 72, 24, 5), (40007, 72, 64, 128, 3), (40000, 64, 136, 16, 30),
                                       (6007, 64, 72, 16, 16), (16385, 64, 64, 8, 9), (16384, 64, 64, 8, 1024),
                                       (9001, 64, 64, 64, 1025)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_lora(S, K, N, r, n, dtype, out_dtype, order):
    g = gen(S + K + r)
    c = lora_case(g, S, K, N, r, n, dtype, out_dtype)
    ids = torch.randint(-2, n + 2, (S,), generator=g, device="cuda").int()       # outside [0, n): none
    if order == "runs":
        ids = ids.sort().values
    ref = lora_ref(c, ids)
    y, u = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids, scale=c["scale"], keep=True)
    assert y.dtype is out_dtype and u.dtype is dtype
    bar = lora_bar(*ref[:3], K, r, dtype, out_dtype, S <= 64)
    within(y, ref[0], bar)
    none = (ids < 0) | (ids >= n)
    assert torch.equal(y[none], c["base"][none]) and (u[none] == 0).all()
    ub = torch.zeros_like(ref[3])
    for e in range(n):
        rows = ids == e
        ub[rows] = c["scale"][e].double() * (c["x"][rows].double().abs() @ c["a"][e].double().abs().T)
    # rounded, and the rest: half an ulp of half an ulp is left
    within(u[:, 0], ref[3], H[dtype] * ref[3].abs() + (2 * K + 40) * U * ub + TINY[dtype])
    within(u[:, 0].double() + u[:, 1].double(), ref[3], H[dtype] ** 2 * ref[3].abs() + (2 * K + 40) * U * ub + TINY[dtype])
    # in place, without a base, without a scale, and the same bits each time
    assert torch.equal(B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids, scale=c["scale"]), y)
    into = c["base"].clone()
    B.situ_moe_lora(into, c["x"], c["a"], c["b"], ids=ids, scale=c["scale"], out=into)
    assert torch.equal(into, y)
    zero = torch.zeros_like(c["base"])
    bare = B.situ_moe_lora(None, c["x"], c["a"], c["b"], ids=ids, out=torch.empty_like(zero))
    assert torch.equal(bare, B.situ_moe_lora(zero, c["x"], c["a"], c["b"], ids=ids, scale=torch.ones(n, device="cuda")))


@pytest.mark.parametrize("S", [40, 500])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_lora_rows_by_offsets(S, dtype):
    g = gen(S)
    n, K, N, r = 6, 264, 200, 16
    c = lora_case(g, S, K, N, r, n, dtype, dtype)
    cuts = torch.randint(0, S + 1, (n - 1,), generator=g, device="cuda").sort().values.int()
    off = torch.cat((torch.tensor([2], device="cuda"), cuts.clamp(min=2), torch.tensor([S - 1], device="cuda"))).int()
    off = torch.cummax(off, 0).values.int()
    e, held = expert_rows(off, S)
    ids = torch.where(held, e, -1).int()
    want = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids, scale=c["scale"])
    assert torch.equal(B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], offsets=off, scale=c["scale"]), want)


@pytest.mark.parametrize("S,n", [(50, 5), (400, 5), (1500, 20)])
def test_lora_rows_do_not_touch_each_other(S, n):
    # an adapter of NaN and infinities, and rows of them, in the same tiles as others
    g = gen(S)
    K, N, r = 136, 264, 24
    c = lora_case(g, S, K, N, r, n, BF16, BF16)
    ids = torch.randint(0, n, (S,), generator=g, device="cuda").int()
    want = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids)
    c["a"][2, 3], c["b"][2, 7] = float("nan"), float("inf")
    c["a"][4], c["b"][4] = float("inf"), float("nan")
    c["x"][ids == 2] = float("inf")
    got = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids)
    fine = (ids != 2) & (ids != 4)
    assert torch.equal(got[fine], want[fine]) and torch.isnan(got[~fine]).all()


@pytest.mark.parametrize("S", [9, 300])
def test_lora_f16_sums_beyond_f16(S):
    # u of 2^20 and more, brought back by small b; and u far below f16's range
    g = gen(S)
    K, N, r = 512, 72, 16
    x, a = normal(g, S, K, std=30.0, dtype=F16), normal(g, 1, r, K, std=3e3, dtype=F16)
    b = normal(g, 1, N, r, std=2e-6, dtype=F16)
    ids = torch.zeros(S, dtype=torch.int32, device="cuda")
    for f in (1.0, 2.0 ** -60):
        c = dict(x=x, a=a, b=b, base=torch.zeros(S, N, device="cuda"), scale=torch.tensor([f], device="cuda"))
        y = B.situ_moe_lora(c["base"], x, a, b, ids=ids, scale=c["scale"])
        ref = lora_ref(c, ids)
        assert ref[3].abs().max() > 2.0 ** 20 * f
        within(y, ref[0], lora_bar(*ref[:3], K, r, F16, F32, False))


def test_lora_layouts_and_nothing():
    g = gen(3)
    for S in (20, 200):
        n, K, N, r = 4, 72, 136, 16
        c = lora_case(g, S, K, N, r, n, BF16, BF16)
        ids = torch.randint(0, n, (S,), generator=g, device="cuda").int()
        want = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids)
        wide = torch.zeros(S, K + 24, dtype=BF16, device="cuda")
        for skip in (0, 8, 3):
            wide[:, skip:skip + K] = c["x"]
            assert torch.equal(B.situ_moe_lora(c["base"], wide[:, skip:skip + K], c["a"], c["b"], ids=ids), want)
        out = torch.full((S, N + 8), 3.0, dtype=BF16, device="cuda")
        B.situ_moe_lora(c["base"].t().contiguous().t(), c["x"], c["a"].transpose(1, 2).contiguous().transpose(1, 2), c["b"],
                        ids=ids.repeat_interleave(2)[::2], out=out[:, :N])
        assert torch.equal(out[:, :N], want) and (out[:, N:] == 3).all()
        empty = B.situ_moe_lora(c["base"][:0], c["x"][:0], c["a"], c["b"], ids=ids[:0])
        assert empty.shape == (0, N)
        none = torch.full_like(ids, -1)
        assert torch.equal(B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=none), c["base"])
        assert (B.situ_moe_lora(None, c["x"], c["a"], c["b"], ids=none) == 0).all()
    with pytest.raises(ValueError):
        B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"])
    with pytest.raises(ValueError):
        B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids, offsets=offsets_of([S, 0, 0, 0]))
    with pytest.raises(ValueError):
        B.situ_moe_lora(c["base"].half(), c["x"], c["a"], c["b"], ids=ids)
    with pytest.raises(ValueError):
        B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], ids=ids.cpu())
    with pytest.raises(B.SituError):
        B.situ_moe_lora(c["base"], c["x"], c["a"][:, :12].contiguous(), c["b"][..., :12].contiguous(), ids=ids)


@pytest.mark.parametrize("counts,spare,K,N,r", [([1], 0, 8, 8, 8), ([40], 3, 72, 136, 8), ([100, 0, 33], 0, 264, 200, 16),
                                                ([700, 200], 5, 136, 392, 24), ([513], 0, 520, 1032, 64),
                                                ([64] * 9, 0, 64, 128, 128)])
@pytest.mark.parametrize("dtype,dx_dtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
def test_lora_gradients(counts, spare, K, N, r, dtype, dx_dtype):
    g = gen(K + N + r)
    S, n, off = sum(counts) + spare, len(counts), offsets_of(counts)
    c = lora_case(g, S, K, N, r, n, dtype, dtype)
    dy, dx0 = normal(g, S, N, std=0.1, dtype=dtype), normal(g, S, K, std=0.1, dtype=dx_dtype)
    _, u = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], offsets=off, scale=c["scale"], keep=True)
    dx, da, db = B.situ_moe_lora_backward(dy, c["x"], c["a"], c["b"], off, u, scale=c["scale"], dx=dx0)
    assert dx.dtype is dx_dtype and da.dtype is dtype and db.dtype is dtype
    h = H[dtype]
    for e in range(n):
        rows = slice(int(off[e]), int(off[e + 1]))
        L = counts[e]
        f, a, b = c["scale"][e].double(), c["a"][e].double(), c["b"][e].double()
        x, d = c["x"][rows].double(), dy[rows].double()
        v, va = f * (d @ b), f * (d.abs() @ b.abs())
        ue, ua = f * (x @ a.T), f * (x.abs() @ a.abs().T)
        want = dx0[rows].double() + v @ a
        v16 = h if dx_dtype is not F32 else 2.0 ** -21
        within(dx[rows], want, H[dx_dtype] * want.abs() + (2 * N + 40) * U * (va @ a.abs())
               + (v16 + (6 * r + 8) * U) * (v.abs() @ a.abs()) + TINY[dx_dtype])
        # u and v in two terms, sums over the rows (16-bit results: by a tenth of half an ulp more), one rounding
        for got, p, pa, t in ((da[e], v, va, x), (db[e].T, ue, ua, d)):
            terms = p.abs().T @ t.abs()
            want = p.T @ t
            within(got, want, 1.2 * h * want.abs() + (h * h + 2 * L * U) * terms + (2 * max(K, N) + 40) * U * (pa.T @ t.abs())
                   + TINY[dtype] * (1 + (t.abs().sum(0)[None] if len(t) else 0)))
    assert torch.equal(dx[sum(counts):], dx0[sum(counts):])
    # into the given gradient, and without one
    into = dx0.clone()
    got = B.situ_moe_lora_backward(dy, c["x"], c["a"], c["b"], off, u, scale=c["scale"], dx=into, out=into)
    assert got[0] is into and torch.equal(into, dx) and torch.equal(got[1], da) and torch.equal(got[2], db)
    bare = B.situ_moe_lora_backward(dy, c["x"], c["a"], c["b"], off, u, scale=c["scale"])[0]
    assert bare.dtype is dtype and (bare[sum(counts):] == 0).all()


@pytest.mark.parametrize("counts,K,N,r", [([1] * 40 + [0] * 20 + [3] * 30, 64, 72, 8), ([63, 64, 65, 0, 127, 128, 129], 136, 64, 40),
                                          ([2000, 0, 3, 700], 1160, 2056, 16), ([5], 8, 4104, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_lora_gradients_of_many_and_ragged_adapters(counts, K, N, r, dtype):
    # rows before the first and after the last adapter's hold NaN
    g = gen(sum(counts) + K)
    S, n = sum(counts) + 9, len(counts)
    off = offsets_of(counts) + 4
    x, dy = normal(g, S, K, dtype=dtype), normal(g, S, N, std=0.1, dtype=dtype)
    a, b = normal(g, n, r, K, std=K ** -0.5, dtype=dtype), normal(g, n, N, r, std=r ** -0.5, dtype=dtype)
    x[:4], x[-5:], dy[:4], dy[-5:] = float("nan"), float("inf"), float("inf"), float("nan")
    _, u = B.situ_moe_lora(None, x, a, b, offsets=off, keep=True)
    dx, da, db = B.situ_moe_lora_backward(dy, x, a, b, off, u)
    v = B.situ_moe_lora(None, dy, b.transpose(1, 2).contiguous(), a.transpose(1, 2).contiguous(), offsets=off, keep=True)[1]
    assert (dx[:4] == 0).all() and (dx[-5:] == 0).all() and torch.isfinite(dx).all()
    # v as the backward pass has it: the same sums by another kernel, so off by the second term's rounding at most
    for e in range(n):
        rows = slice(int(off[e]), int(off[e + 1]))
        L = counts[e]
        for got, p, t in ((da[e], v[rows].double().sum(1), x[rows].double()),
                          (db[e].T, u[rows].double().sum(1), dy[rows].double())):
            want, terms = p.T @ t, p.abs().T @ t.abs()
            within(got, want, 1.2 * H[dtype] * want.abs() + (2 * H[dtype] ** 2 + 2 * L * U + 2 * max(K, N) * U) * terms
                   + TINY[dtype] * (1 + (t.abs().sum(0)[None] if L else 0)))
            if L == 0:
                assert (got == 0).all()
    again = B.situ_moe_lora_backward(dy, x, a, b, off, u)
    assert torch.equal(again[0], dx) and torch.equal(again[1], da) and torch.equal(again[2], db)


def test_lora_gradients_of_long_f16_sums():
    # more rows than one sum of f16 results takes, and terms of one sign
    S, C, r = 9000, 10240, 8
    g = gen(77)
    x, dy = torch.rand(S, C, generator=g, device="cuda").half(), (torch.rand(S, C, generator=g, device="cuda") * 0.01).half()
    a, b = torch.full((1, r, C), 1e-3, device="cuda").half(), torch.full((1, C, r), 1e-2, device="cuda").half()
    off = torch.tensor([0, S], dtype=torch.int32, device="cuda")
    _, u = B.situ_moe_lora(None, x, a, b, offsets=off, keep=True)
    _, da, db = B.situ_moe_lora_backward(dy, x, a, b, off, u)
    want = dy.double().T[:512] @ u.double().sum(1)
    # the rounding, a tenth of it more, and 2 U a term of the sums of a chunk of 512
    within(db[0, :512], want, (1.1 * H[F16] + 512 * 2 * U + 20 * U) * want)


def test_lora_linear_by_autograd():
    g = gen(8)
    counts, K, N, r = [60, 0, 41], 64, 128, 8
    off = offsets_of(counts)
    c = lora_case(g, 101, K, N, r, 3, BF16, F32)
    leaves = [c[k].clone().requires_grad_() for k in ("base", "x", "a", "b")]
    y = B.lora_linear(*leaves, off, c["scale"])
    dy = normal(g, 101, N, std=0.1, dtype=BF16).float()      # exact in bf16
    y.backward(dy)
    ref = [t.detach().double().requires_grad_() for t in leaves]
    want = ref[0].clone()
    for e in range(3):
        rows = slice(int(off[e]), int(off[e + 1]))
        want[rows] = ref[0][rows] + c["scale"][e].double() * (ref[1][rows] @ ref[2][e].T) @ ref[3][e].T
    want.backward(dy.double())
    assert torch.equal(leaves[0].grad, dy)
    # a rounding of the result, and of v or u on the way to x's gradient
    for got, r_ in zip(leaves[1:], ref[1:]):
        assert (got.grad.double() - r_.grad).norm() <= 2 * H[BF16] * r_.grad.norm()
    y = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], offsets=off, scale=c["scale"])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(B.lora_linear(*leaves, off, c["scale"]).sum(), leaves[1], create_graph=True)[0].sum().backward()


def test_lora_gradients_without_rows():
    a, b = torch.randn(3, 8, 64, device="cuda").bfloat16(), torch.randn(3, 72, 8, device="cuda").bfloat16()
    z = lambda c: torch.zeros(0, c, dtype=BF16, device="cuda")  # noqa: E731
    dx, da, db = B.situ_moe_lora_backward(z(72), z(64), a, b, torch.zeros(4, dtype=torch.int32, device="cuda"), z(16).view(0, 2, 8))
    assert dx.shape == (0, 64) and (da == 0).all() and (db == 0).all()


# --------------------------------------------------------------------------
# together, streams, graphs
# --------------------------------------------------------------------------

@pytest.mark.parametrize("keep", ["mxfp8", "16bit"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_expert_ffn(keep, dtype):
    g = gen(6)
    counts, Hd, I = [40, 0, 77, 11], 136, 72
    S, E, off = sum(counts) + 4, 4, offsets_of(counts)
    p0, p1 = torch.full((E,), 1.5, device="cuda"), torch.full((E,), 2.0, device="cuda")
    x, w1, w2 = normal(g, S, Hd, dtype=dtype), normal(g, E, 2 * I, Hd, std=Hd ** -0.5, dtype=dtype), normal(
        g, E, Hd, I, std=I ** -0.5, dtype=dtype)
    leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
    y = B.expert_ffn(*leaves, off, p0, p1, keep=keep)
    dy = normal(g, S, Hd, std=0.2, dtype=dtype)
    y.backward(dy)
    ref = [t.double().requires_grad_() for t in (x, w1, w2)]
    want = torch.zeros(S, Hd, dtype=F64, device="cuda")
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        gg, u = (ref[0][rows] @ ref[1][e].T).chunk(2, 1)
        want[rows] = (1.5 * torch.tanh(gg / 1.5) * torch.sigmoid(gg) * 2 * torch.tanh(u / 2)) @ ref[2][e].T
    want.backward(dy.double())
    # forward: 16-bit roundings of gate/up and h, the result's.  Backward: the kept values are off by 2^-4 relative each
    # (2^-5 on average), through derivatives of order one; 2^-3 bounds the norm
    assert (y.double() - want).norm() <= 6 * H[dtype] * want.norm()
    for got, r in zip(leaves, ref):
        assert (got.grad.double() - r.grad).norm() <= 2.0 ** -3 * r.grad.norm()
    # what the gradients are, from the calls that make them
    gate_up = B.situ_moe_grouped_gemm(x, w1, off)
    h, q, s = B.situ_moe_gated(gate_up, p0, p1, off, save=True)
    d, h2 = B.situ_moe_gated_backward(B.situ_moe_grouped_gemm_dgrad(dy, w2, off), q, s, p0, p1, off, want_h=True)
    xk = x if keep == "16bit" else B.situ_moe_restore_mxfp8(*B.situ_moe_save_mxfp8(x), dtype)
    assert torch.equal(leaves[0].grad, B.situ_moe_grouped_gemm_dgrad(d, w1, off))
    assert torch.equal(leaves[1].grad, B.situ_moe_grouped_gemm_wgrad(d, xk, off))
    assert torch.equal(leaves[2].grad, B.situ_moe_grouped_gemm_wgrad(dy, h2, off))
    # frozen weights cost nothing of theirs
    only = x.clone().requires_grad_()
    B.expert_ffn(only, w1, w2, off, p0, p1, keep=keep).backward(dy)
    assert torch.equal(only.grad, leaves[0].grad)


def step(S=300, seed=1):
    """One of each operator's calls, and their results."""
    g = gen(seed)
    E, k, K, N, r = 40, 4, 136, 264, 16
    logits, dw = router_case(S, E, k, seed)
    ids, w = B.situ_moe_route_topk(logits, k)
    one = torch.ones((), device="cuda")
    gate_up, dh = normal(g, S, 2 * K), normal(g, S, K)
    off = offsets_of([S // 3] * 3)
    p0, p1 = caps(g, 3, SITU)
    c = lora_case(g, S, K, N, r, 3, BF16, BF16)
    dy = normal(g, S, N, std=0.1)
    few = torch.arange(30, device="cuda").int() % 3

    def run(stream=None):
        kw = dict(stream=stream)
        loss, counts, tokens, stats = B.situ_moe_balance_loss(logits, ids, **kw)
        d = B.situ_moe_router_backward(logits, ids, counts, tokens, stats, dloss=one, topk_weights=w, dweights=dw, **kw)
        h, q, s = B.situ_moe_gated(gate_up, p0, p1, off, save=True, **kw)
        dx, _ = B.situ_moe_gated_backward(dh, q, s, p0, p1, off, **kw)
        xk = B.situ_moe_restore_mxfp8(*B.situ_moe_save_mxfp8(h, **kw), BF16, **kw)
        y, u = B.situ_moe_lora(c["base"], xk, c["a"], c["b"], offsets=off, scale=c["scale"], keep=True, **kw)
        back = B.situ_moe_lora_backward(dy, xk, c["a"], c["b"], off, u, scale=c["scale"], dx=dh, **kw)
        row = B.situ_moe_lora(y[:30], xk[:30], c["a"], c["b"], ids=few, **kw)
        return [loss, counts, tokens, d, h, q, s, dx, xk, y, u, *back, row]

    return run, (logits, gate_up, dh, dy)


def test_streams():
    run, _ = step()
    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(stream=s)
    with torch.cuda.stream(s):
        again = run()
    s.synchronize()
    for a, b, c in zip(want, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_and_replayed_on_new_inputs():
    run, inputs = step()
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in (2, 3):
        other, values = step(seed=seed)
        for t, v in zip(inputs, values):
            t.copy_(v)
        want = run()
        for t in got:
            t.zero_()
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_a_training_step_captured_and_replayed():
    g = gen(5)
    T, Hd, I, E, r, k = 120, 64, 40, 6, 8, 2
    x = normal(g, T, Hd)
    router = (torch.randn(Hd, E, generator=g, device="cuda") * Hd ** -0.5).requires_grad_()
    w1, w2 = normal(g, E, 2 * I, Hd, std=Hd ** -0.5).requires_grad_(), normal(g, E, Hd, I, std=I ** -0.5).requires_grad_()
    a, b = normal(g, E, r, Hd, std=Hd ** -0.5).requires_grad_(), normal(g, E, Hd, r, std=0.3).requires_grad_()
    p0, p1 = torch.full((E,), 1.5, device="cuda"), torch.full((E,), 2.0, device="cuda")
    dy = normal(g, T * k, Hd, std=0.2)

    def run():
        ids, w, counts, loss = B.balanced_route(x.float() @ router, k)
        _, off, slot, _ = B.situ_moe_permute(ids, E, E, 0)
        rows = x[slot.long() // k]
        y = B.lora_linear(B.expert_ffn(rows, w1, w2, off, p0, p1), rows, a, b, off)
        return torch.autograd.grad((y.float() * dy.float()).sum() + loss + (w * w).sum(), (router, w1, w2, a, b))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    x.copy_(normal(g, T, Hd))
    graph.replay()
    for got_, want in zip(got, run()):
        assert torch.equal(got_, want)


def test_a_capture_beside_a_living_graph_of_the_same_leaves_is_refused():
    g = gen(6)
    S, K, N, r = 300, 72, 64, 8
    x, dy = normal(g, S, K), normal(g, S, N)
    a, b = normal(g, 2, r, K).requires_grad_(), normal(g, 2, N, r).requires_grad_()
    off = offsets_of([100, 200])

    def run():
        a.grad = b.grad = None
        y = B.lora_linear(torch.zeros(S, N, dtype=BF16, device="cuda"), x, a, b, off)
        return y, a, b

    y = run()[0]                                    # a living graph, of the current stream
    again = run()[0]                                # another beside it is fine
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="alive"):
        with torch.cuda.graph(graph):
            run()
    again.backward(dy)
    want = a.grad.clone(), b.grad.clone()
    del y, again
    a.grad = b.grad = None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()[0].backward(dy)
    graph.replay()
    assert torch.equal(a.grad, want[0]) and torch.equal(b.grad, want[1])


def test_no_work_after_a_wait_was_given_up():
    g = gen(7)
    S, K, N, r, n = 300, 72, 136, 16, 3
    c = lora_case(g, S, K, N, r, n, BF16, BF16)
    off, dy = offsets_of([100] * 3), normal(g, S, N)
    _, u = B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], offsets=off, keep=True)
    want = B.situ_moe_lora_backward(dy, c["x"], c["a"], c["b"], off, u)
    out, dx = torch.full((S, N), 3.0, dtype=BF16, device="cuda"), torch.full((S, K), 3.0, dtype=BF16, device="cuda")
    B._status_word(torch.cuda.current_device()).fill_(99)
    try:
        B.situ_moe_lora(c["base"], c["x"], c["a"], c["b"], offsets=off, out=out)
        B.situ_moe_lora_backward(dy, c["x"], c["a"], c["b"], off, u, out=dx)
        assert (out == 3).all() and (dx == 3).all()
    finally:
        assert B.situ_moe_gemm_status(reset=True) == 99
    for a, b in zip(B.situ_moe_lora_backward(dy, c["x"], c["a"], c["b"], off, u), want):
        assert torch.equal(a, b)


def test_two_graphs_and_eager_calls_in_turn():
    runs = [step(S=s, seed=s)[0] for s in (90, 240)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    graphs, got = [], []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(r())
        graphs.append(graph)
    for _ in range(3):
        for graph, r in zip(graphs, runs):
            graph.replay()
            r()
    for g_, w_ in zip(got, want):
        for a, b in zip(g_, w_):
            assert torch.equal(a, b)


def test_far_offsets():
    # elements past 2^31: the last rows of large operands
    S, I = 33000, 32768
    x = torch.zeros(S, 2 * I, dtype=BF16, device="cuda")
    g = gen(2)
    x[-40:] = normal(g, 40, 2 * I)
    one = torch.ones(1, device="cuda")
    h, q, s = B.situ_moe_gated(x, one, one, save=True)
    h1, q1, s1 = B.situ_moe_gated(x[-40:].clone(), one, one, save=True)
    assert torch.equal(h[-40:], h1) and torch.equal(q[-40:], q1) and torch.equal(s[-40:], s1)
    dh = torch.ones(S, I, dtype=BF16, device="cuda")
    dx, _ = B.situ_moe_gated_backward(dh, q, s, one, one)
    assert torch.equal(dx[-40:], B.situ_moe_gated_backward(dh[-40:].clone(), q1, s1, one, one)[0])
    del h, q, s, dh, dx
    a, b = normal(g, 2, 16, 2 * I, std=0.01), normal(g, 2, 136, 16)
    ids = torch.arange(S, device="cuda").int() % 2
    y = B.situ_moe_lora(None, x, a, b, ids=ids)
    assert (y[:-40] == 0).all()
    d = (B.situ_moe_lora(None, x[-64:].clone(), a, b, ids=ids[-64:]) - y[-64:]).double()
    assert d.norm() <= 4 * H[BF16] * y[-64:].double().norm()
    wide = B.situ_moe_lora(None, torch.ones(S, 8, dtype=BF16, device="cuda"), normal(g, 1, 8, 8), normal(g, 1, 2 * I, 8),
                           ids=torch.zeros(S, dtype=torch.int32, device="cuda"))
    assert (wide == wide[0]).all()
