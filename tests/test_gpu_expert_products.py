"""The expert products with 16-bit and with E4M3 weights, on the GPU, against
plain sums in 64 bits.

Bars, derived before any run.  A sum of L products kept in fp32 in any order,
each addition rounded or truncated, is off by at most L * 2^-23 * sum |a b|
(every addition loses at most 2^-23 of a partial sum, which is at most the sum
of magnitudes); the E4M3 product adds a few roundings per block of 128, far
fewer than L.  The one rounding to the output type adds half a unit in the
last place: 2^-8 (bf16), 2^-11 (f16) or 2^-24 (fp32) of the value, or half the
spacing of f16's subnormals.  Quantisation codes and scales are exact.
"""
import ctypes

import numpy as np
import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()
    yield
    assert B.situ_moe_gemm_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offsets_of(counts, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def assert_sum(got, ref, mag, L, dtype):
    """got (dtype) against ref and the sums of magnitudes, both fp64."""
    got, ref, mag = got.double().cpu(), ref.cpu(), mag.cpu()
    bar = (L + 2) * 2.0 ** -23 * mag
    bar = bar + HALF_ULP[dtype] * (ref.abs() + bar) + TINY[dtype]
    worst = ((got - ref).abs() - bar).max().item() if got.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 0.0, worst


def reference(direction, a, b, counts, start, S, N, K):
    """(value, sum of magnitudes) in 64 bits."""
    a, b = a.double().cpu(), b.double().cpu()
    if direction == "wgrad":
        out = torch.zeros(len(counts), N, K, dtype=torch.float64)
        mag = torch.zeros_like(out)
        r = start
        for e, n in enumerate(counts):
            out[e] = a[r:r + n].T @ b[r:r + n]
            mag[e] = a[r:r + n].abs().T @ b[r:r + n].abs()
            r += n
        return out, mag
    out = torch.zeros(S, N if direction == "forward" else K, dtype=torch.float64)
    mag = torch.zeros_like(out)
    r = start
    for e, n in enumerate(counts):
        w = b[e].T if direction == "forward" else b[e]
        out[r:r + n] = a[r:r + n] @ w
        mag[r:r + n] = a[r:r + n].abs() @ w.abs()
        r += n
    return out, mag


def call(direction, a, b, offsets, **kw):
    f = {"forward": B.situ_moe_grouped_gemm, "dgrad": B.situ_moe_grouped_gemm_dgrad,
         "wgrad": B.situ_moe_grouped_gemm_wgrad}[direction]
    return f(a, b, offsets, **kw)


def operands(direction, g, S, E, N, K, dtype):
    if direction == "forward":
        return normal(g, S, K, dtype=dtype), normal(g, E, N, K, dtype=dtype, std=0.1), K
    if direction == "dgrad":
        return normal(g, S, N, dtype=dtype), normal(g, E, N, K, dtype=dtype, std=0.1), N
    return normal(g, S, N, dtype=dtype), normal(g, S, K, dtype=dtype), S


GROUPS = [
    dict(counts=[1], start=0, spare=0),
    dict(counts=[0, 3, 0, 1, 17, 0], start=0, spare=5),                # short groups, empty ones at both ends
    dict(counts=[16, 15, 64, 63, 65, 1, 0, 32, 33], start=3, spare=2),  # about 32 rows each: either side of a stage
    dict(counts=[100, 0, 31, 130], start=0, spare=0),
    dict(counts=[127, 128, 129, 70, 1], start=1, spare=1),
    dict(counts=[256, 300, 0, 257], start=0, spare=9),
    dict(counts=[700], start=0, spare=0),
    dict(counts=[0, 0, 0], start=0, spare=7),                          # no row has an expert
]
SHAPES = [(8, 8), (24, 72), (128, 64), (136, 264), (264, 136), (1000, 200), (64, 520)]


@pytest.mark.parametrize("direction", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("grp", range(len(GROUPS)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_grouped_matches_64_bit_sums(direction, grp, shape):
    c = GROUPS[grp]
    N, K = SHAPES[shape]
    counts, start = c["counts"], c["start"]
    S = start + sum(counts) + c["spare"]
    # types in turn over the grid
    dtype = (torch.bfloat16, torch.float16)[(grp + shape) % 2]
    out_dtype = (dtype, torch.float32)[(grp // 2 + shape) % 2]
    a, b, L = operands(direction, gen(grp * 100 + shape), S, len(counts), N, K, dtype)
    got = call(direction, a, b, offsets_of(counts, start), out_dtype=out_dtype)
    ref, mag = reference(direction, a, b, counts, start, S, N, K)
    assert got.dtype == out_dtype
    assert_sum(got, ref, mag, L, out_dtype)


def test_many_experts():
    g = gen(5)
    rng = np.random.default_rng(1)
    counts = (rng.integers(0, 4, 1024) * (rng.random(1024) < 0.5)).tolist()
    S, N, K = sum(counts), 40, 88
    for direction in ("forward", "dgrad", "wgrad"):
        a, b, L = operands(direction, g, S, 1024, N, K, torch.bfloat16)
        got = call(direction, a, b, offsets_of(counts), out_dtype=torch.float32)
        ref, mag = reference(direction, a, b, counts, 0, S, N, K)
        assert_sum(got, ref, mag, L, torch.float32)


@pytest.mark.parametrize("counts", [[40, 17, 0, 3], [300, 129, 0, 260]])
def test_wide_persistent_walk(counts):
    # more tiles than CTAs, and long contractions over every ring stage
    N, K = 2056, 1544
    S = sum(counts)
    for direction in ("forward", "dgrad", "wgrad"):
        a, b, L = operands(direction, gen(3), S, len(counts), N, K, torch.bfloat16)
        got = call(direction, a, b, offsets_of(counts))
        ref, mag = reference(direction, a, b, counts, 0, S, N, K)
        assert_sum(got, ref, mag, L, torch.bfloat16)


# one case per kernel form, by the rules on sizes (a GPU of 152 SMs): tiles of
# 32, 64 and 128 tokens whose contraction is split over a cluster, with odd
# shares of the stages; 128 and 256 tokens unsplit; a single CTA at 256 tokens
# (M side of at most 128)
FORMS = [([5], 136, 2056), ([5, 0, 20], 264, 2056), ([50], 200, 1032), ([90], 136, 1544), ([44, 40, 0, 30], 72, 1100 // 4 * 8),
         ([90, 60, 0, 97, 80, 70, 88, 99], 1416, 200), ([150, 300, 0, 260, 129, 1, 90], 2056, 136),
         ([700, 5, 900], 2312, 72), ([16000], 128, 128), ([9000, 0, 10000], 72, 120)]


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("direction", ["forward", "dgrad"])
def test_every_form_of_the_grouped_product(form, direction):
    counts, M, L = FORMS[form]
    N, K = (M, L) if direction == "forward" else (L, M)
    S = 1 + sum(counts) + 2
    dtype = (torch.bfloat16, torch.float16)[form % 2]
    a, b, L = operands(direction, gen(form), S, len(counts), N, K, dtype)
    for out_dtype in (dtype, torch.float32):
        got = call(direction, a, b, offsets_of(counts, 1), out_dtype=out_dtype)
        ref, mag = reference(direction, a, b, counts, 1, S, N, K)
        assert_sum(got, ref, mag, L, out_dtype)


@pytest.mark.parametrize("counts,N,K", [([3000], 152, 264), ([1700, 0, 5, 900, 64, 63], 136, 72), ([5000, 1], 8, 8),
                                        ([700, 1500], 264, 520), ([9999], 1000, 72)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_split_over_rows(counts, N, K, accumulate):
    # few output tiles: a cluster takes one tile, each CTA some of the rows;
    # groups with fewer stages than CTAs, and with none
    S = 3 + sum(counts) + 1
    dy, x, L = operands("wgrad", gen(N), S, len(counts), N, K, torch.bfloat16)
    x[:3] = float("nan")
    dy[-1:] = float("inf")
    old = normal(gen(1), len(counts), N, K, dtype=torch.float32)
    off = offsets_of(counts, 3)
    ref, mag = reference("wgrad", dy, x, counts, 3, S, N, K)
    for out_dtype in (torch.bfloat16, torch.float32):
        out = old.to(out_dtype)
        o = out.double().cpu() if accumulate else 0.0
        got = B.situ_moe_grouped_gemm_wgrad(dy, x, off, out=out, accumulate=accumulate)
        assert_sum(got, ref + o, mag + abs(o), L, out_dtype)
        again = old.to(out_dtype)
        B.situ_moe_grouped_gemm_wgrad(dy, x, off, out=again, accumulate=accumulate)
        assert torch.equal(again, got)


@pytest.mark.parametrize("direction", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [[5, 0, 18, 1, 40], [200, 0, 333, 70]])
def test_infinities_and_nans_stay_in_their_group(direction, counts):
    # every second expert's rows (and the rows of none) hold infinities and
    # NaNs, and so do its weights: the others' results do not change
    E, N, K, start = len(counts), 72, 200, 2
    S = start + sum(counts) + 3
    a, b, L = operands(direction, gen(11), S, E, N, K, torch.bfloat16)
    off = offsets_of(counts, start)
    bad = torch.ones(S, dtype=torch.bool)
    r = start
    for e, n in enumerate(counts):
        bad[r:r + n] = e % 2 == 1
        r += n
    poison = torch.tensor([float("inf"), float("nan"), -float("inf")], device="cuda", dtype=a.dtype)
    a2, b2 = a.clone(), b.clone()
    a2[bad.cuda()] = poison[torch.arange(a.shape[1], device="cuda") % 3]
    if direction == "wgrad":
        b2[bad.cuda()] = poison[torch.arange(b.shape[1], device="cuda") % 3]
    else:
        b2[1::2] = float("nan")
    got = call(direction, a2, b2, off)
    a[bad.cuda()] = 0
    ref, mag = reference(direction, a, b, counts, start, S, N, K)
    if direction == "wgrad":
        for e in range(0, E, 2):
            assert_sum(got[e], ref[e], mag[e], L, got.dtype)
    else:
        keep = ~bad
        assert_sum(got[keep.cuda()], ref[keep], mag[keep], L, got.dtype)
        ends = torch.cat([torch.arange(start), torch.arange(S - 3, S)])
        assert (got[ends.cuda()] == 0).all()


def test_rows_of_no_expert_are_zeroed_or_left():
    counts, S, N, K = [3, 9], 20, 64, 128
    g = gen(2)
    x, w, dy = normal(g, S, K), normal(g, 2, N, K), normal(g, S, N)
    off = offsets_of(counts, 4)
    for f, first in ((B.situ_moe_grouped_gemm, x), (B.situ_moe_grouped_gemm_dgrad, dy)):
        out = torch.full((S, N if first is x else K), 7.0, dtype=torch.bfloat16, device="cuda")
        f(first, w, off, out=out)
        assert (out[:4] == 0).all() and (out[16:] == 0).all() and (out[4:16] != 0).any()
        kept = torch.full_like(out, 7.0)
        f(first, w, off, out=kept, zero_rest=False)
        assert (kept[:4] == 7).all() and (kept[16:] == 7).all() and torch.equal(kept[4:16], out[4:16])


def test_strided_rows_and_copied_layouts():
    counts, N, K = [33, 0, 50], 72, 136
    S = sum(counts)
    g = gen(4)
    off = offsets_of(counts)
    xw, dyw = normal(g, S, K + 64), normal(g, S, N + 24)
    w = normal(g, 3, N, K, std=0.1)
    for x, dy in ((xw[:, 16:16 + K], dyw[:, 8:8 + N]),                                # read in place
                  (xw[:, 3:3 + K], dyw[:, 1:1 + N]),                                  # misaligned: copied
                  (normal(g, K, S).T, normal(g, N, S).T),                             # column-major: copied
                  (normal(g, 1, K).expand(S, K), normal(g, 1, N).expand(S, N))):      # broadcast: copied
        out = torch.zeros(S, N + 40, dtype=torch.bfloat16, device="cuda")
        y = B.situ_moe_grouped_gemm(x, w, off, out=out[:, 8:8 + N])
        assert (out[:, :8] == 0).all() and (out[:, 8 + N:] == 0).all()
        assert_sum(y, *reference("forward", x, w, counts, 0, S, N, K), K, torch.bfloat16)
        dx = B.situ_moe_grouped_gemm_dgrad(dy, w, off)
        assert_sum(dx, *reference("dgrad", dy, w, counts, 0, S, N, K), N, torch.bfloat16)
        dw = B.situ_moe_grouped_gemm_wgrad(dy, x, off)
        assert_sum(dw, *reference("wgrad", dy, x, counts, 0, S, N, K), S, torch.bfloat16)
    wt = normal(g, 3, K, N, std=0.1).transpose(1, 2)                                  # weights stored [E, K, N]
    y = B.situ_moe_grouped_gemm(xw[:, :K], wt, off)
    assert_sum(y, *reference("forward", xw[:, :K], wt, counts, 0, S, N, K), K, torch.bfloat16)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16])
def test_weight_gradient_accumulates(out_dtype):
    counts, N, K = [20, 0, 77], 136, 72
    S = sum(counts)
    g = gen(6)
    dy, x = normal(g, S, N, dtype=torch.float16), normal(g, S, K, dtype=torch.float16)
    old = normal(g, 3, N, K, dtype=out_dtype, std=5.0)
    out = old.clone()
    got = B.situ_moe_grouped_gemm_wgrad(dy, x, offsets_of(counts), out=out, accumulate=True)
    assert got is out and torch.equal(out[1], old[1])
    ref, mag = reference("wgrad", dy, x, counts, 0, S, N, K)
    assert_sum(out, ref + old.double().cpu(), mag + old.double().cpu().abs(), S, out_dtype)


def test_no_rows():
    w = torch.ones(2, 64, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    off = offsets_of([0, 0])
    assert B.situ_moe_grouped_gemm(x, w, off).shape == (0, 64)
    dw = torch.full((2, 64, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    B.situ_moe_grouped_gemm_wgrad(x, x, off, out=dw, accumulate=True)
    assert (dw == 3).all()
    B.situ_moe_grouped_gemm_wgrad(x, x, off, out=dw)
    assert (dw == 0).all()


def test_bad_offsets_stay_inside_the_operands():
    # offsets past S and descending ones are clamped: no fault, and a group
    # that is intact keeps its result
    S, N, K = 50, 64, 64
    g = gen(9)
    x, w, dy = normal(g, S, K), normal(g, 4, N, K), normal(g, S, N)
    off = torch.tensor([0, 10, 5, 2000000000, 60], dtype=torch.int32, device="cuda")
    y = B.situ_moe_grouped_gemm(x, w, off)
    B.situ_moe_grouped_gemm_dgrad(dy, w, off)
    dw = B.situ_moe_grouped_gemm_wgrad(dy, x, off)
    ref, mag = reference("wgrad", dy[:10], x[:10], [10], 0, 10, N, K)
    assert_sum(dw[:1], ref, mag, 10, dw.dtype)
    assert y.shape == (S, N)
    assert B.situ_moe_gemm_status() == 0


def test_another_stream_and_repeat_bits():
    counts, N, K = [60, 200, 0, 140], 512, 640
    S = sum(counts)
    g = gen(12)
    x, w, off = normal(g, S, K), normal(g, 4, N, K, std=0.1), offsets_of(counts)
    dy = normal(g, S, N)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y1 = B.situ_moe_grouped_gemm(x, w, off)
    y2 = B.situ_moe_grouped_gemm(x, w, off, stream=s)
    torch.cuda.synchronize()
    y3 = B.situ_moe_grouped_gemm(x, w, off)
    assert torch.equal(y1, y2) and torch.equal(y1, y3)
    d1, d2 = (B.situ_moe_grouped_gemm_wgrad(dy, x, off, out_dtype=torch.float32) for _ in range(2))
    assert torch.equal(d1, d2)


def test_captured_in_a_graph():
    counts, N, K = [3, 0, 9], 128, 256
    g = gen(13)
    x, w, off = normal(g, 12, K), normal(g, 3, N, K), offsets_of(counts)
    out = B.situ_moe_grouped_gemm(x, w, off)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.situ_moe_grouped_gemm(x, w, off, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# the differentiable product
# ---------------------------------------------------------------------------

def test_grouped_linear_gradients():
    counts, N, K = [40, 0, 3, 150], 64, 96
    S = sum(counts) + 6
    g = gen(21)
    x = normal(g, S, K).requires_grad_()
    w = normal(g, 4, N, K, std=0.1).requires_grad_()
    off = offsets_of(counts)
    y = B.grouped_linear(x, w, off)
    dy = normal(g, S, N)
    y.backward(dy)
    xd, wd = x.detach(), w.detach()
    assert_sum(x.grad, *reference("dgrad", dy, wd, counts, 0, S, N, K), N, torch.bfloat16)
    assert_sum(w.grad, *reference("wgrad", dy, xd, counts, 0, S, N, K), S, torch.bfloat16)
    assert (x.grad[-6:] == 0).all() and (w.grad[1] == 0).all()


def test_grouped_linear_takes_expanded_gradients_and_frozen_operands():
    counts, N, K = [10, 0, 22], 24, 32
    g = gen(23)
    off = offsets_of(counts)
    x, w = normal(g, 32, K), normal(g, 3, N, K, std=0.1).requires_grad_()
    B.grouped_linear(x, w, off).float().sum().backward()          # a broadcast gradient, x frozen
    ones = torch.ones(32, N, dtype=torch.bfloat16, device="cuda")
    assert_sum(w.grad, *reference("wgrad", ones, x, counts, 0, 32, N, K), 32, torch.bfloat16)
    assert x.grad is None
    x.requires_grad_()
    y = B.grouped_linear(x, w.detach(), off)
    y.backward(ones[:1].expand(32, N))
    assert_sum(x.grad, *reference("dgrad", ones, w.detach(), counts, 0, 32, N, K), N, torch.bfloat16)


def test_gradients_against_differences():
    # the product is linear in x and in w, so a central difference is exact up
    # to the sums' own error: with h = 1/4 and values on a grid of 1/8, x +- h d
    # and w +- h d are bf16 numbers
    counts, N, K = [17, 0, 30], 40, 48
    S = sum(counts)
    g = gen(22)
    off = offsets_of(counts)

    def grid(*shape):
        return torch.randint(-8, 9, shape, generator=g, device="cuda").to(torch.bfloat16) / 8

    x, w, dy = grid(S, K), grid(3, N, K), grid(S, N)
    dirx, dirw = torch.sign(grid(S, K)), torch.sign(grid(3, N, K))
    dx = B.situ_moe_grouped_gemm_dgrad(dy, w, off, out_dtype=torch.float32).double()
    dw = B.situ_moe_grouped_gemm_wgrad(dy, x, off, out_dtype=torch.float32).double()
    h = 0.25

    def loss(x_, w_):
        return (B.situ_moe_grouped_gemm(x_, w_, off, out_dtype=torch.float32).double() * dy.double()).sum()

    for slope, diff in (((dx * dirx.double()).sum(), (loss(x + h * dirx, w) - loss(x - h * dirx, w)) / (2 * h)),
                        ((dw * dirw.double()).sum(), (loss(x, w + h * dirw) - loss(x, w - h * dirw)) / (2 * h))):
        # every product is a multiple of 2^-8 below 2^4: all sums are exact in fp32
        assert slope.item() == diff.item()


# ---------------------------------------------------------------------------
# E4M3 with block scales
# ---------------------------------------------------------------------------

def plain_quant(x, rows):
    """Codes and scales in IEEE fp32, block by block."""
    x3 = x.float().cpu().reshape(-1, *x.shape[-2:])
    E, R, K = x3.shape
    nr, nk = -(-R // rows), -(-K // 128)
    q = torch.empty(x3.shape, dtype=torch.float8_e4m3fn)
    s = torch.empty(E, nr, nk)
    for r in range(nr):
        for k in range(nk):
            b = x3[:, r * rows:(r + 1) * rows, k * 128:(k + 1) * 128]
            sc = b.abs().amax((1, 2)) / 448.0
            sc = torch.where(sc < 2.0 ** -126, torch.full_like(sc, 2.0 ** -126), sc)
            s[:, r, k] = sc
            q[:, r * rows:(r + 1) * rows, k * 128:(k + 1) * 128] = (b / sc[:, None, None]).to(torch.float8_e4m3fn)
    return q.reshape(x.shape), s.reshape(*x.shape[:-2], nr, nk)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 8), (7, 128), (64, 136), (129, 1000), (3, 130, 264), (2, 256, 384)])
def test_quant_is_exact(rows, dtype, shape):
    g = gen(sum(shape))
    x = torch.randn(shape, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-6, 7, (*shape[:-1], 1), generator=g, device="cuda").float())
    x.view(-1)[::7] = 0
    x = x.to(dtype)
    q, s = B.situ_moe_quant_fp8(x, rows)
    rq, rs = plain_quant(x, rows)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu().view(torch.float8_e4m3fn).float(), rq.float())


@pytest.mark.parametrize("rows", [1, 128])
def test_quant_extremes(rows):
    x = torch.zeros(rows * 6, 256, device="cuda")
    x[rows:2 * rows, 5] = 2.0 ** -140        # the scale's floor
    x[2 * rows:3 * rows] = 3.4e38
    x[3 * rows, 0] = float("inf")
    x[4 * rows, 1] = float("nan")
    x[5 * rows:, 130] = -2.0 ** -126
    q, s = B.situ_moe_quant_fp8(x, rows)
    v = q.view(torch.float8_e4m3fn).float().cpu()
    rq, rs = plain_quant(x, rows)
    s = s.cpu()
    assert torch.equal(s.isnan(), rs.isnan()) and torch.equal(s[~s.isnan()], rs[~rs.isnan()])
    assert s[3, 0].isinf() and s[4, 0].isnan() and (s[:3].isfinite()).all()
    assert torch.equal(v.isnan(), rq.float().isnan())
    ok = ~v.isnan()
    assert torch.equal(v[ok], rq.float()[ok])
    assert (v[:rows] == 0).all() and (s[0] == 2.0 ** -126).all()


def test_quant_codes_are_those_of_a_correct_division():
    # blocks whose scales have random mantissas, with values at, just below
    # and just above the midpoints between neighbouring codes: a quotient off
    # by one unit in the last place changes a code here
    g = gen(33)
    R = 4096
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = ((grid[1:] + grid[:-1]) / 2).cuda()
    x = torch.zeros(R, 128, device="cuda")
    x[:, 0] = (1 + torch.rand(R, generator=g, device="cuda")) * torch.exp2(
        torch.randint(-70, 100, (R,), generator=g, device="cuda").float())
    scale = x[:, 0].cpu() / 448.0
    v = (mid[:, None] * scale.cuda()).T                  # rounded products: within an ulp of the midpoints
    v = (v.view(torch.int32) + torch.randint(-1, 2, v.shape, generator=g, device="cuda", dtype=torch.int32)).view(
        torch.float32)
    x[:, 1:127] = v
    q, s = B.situ_moe_quant_fp8(x)
    rq, rs = plain_quant(x, 1)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq.view(torch.uint8))


def test_quant_strided_and_out():
    g = gen(31)
    big = normal(g, 40, 400)
    for x in (big[:, 8:8 + 264], big[:, 3:3 + 264], normal(g, 264, 40).T):
        rq, rs = plain_quant(x, 1)
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(40, 3, device="cuda")
        B.situ_moe_quant_fp8(x, 1, out=(q, s))
        assert torch.equal(q.cpu().float(), rq.float()) and torch.equal(s.cpu(), rs)
    q, s = B.situ_moe_quant_fp8(big[:0], 1)
    assert q.shape == (0, 400) and s.shape == (0, 4)


def fp8_operands(g, S, E, N, K, scale_spread=6.0):
    """Random codes (every finite one) and scales over 2^+-scale_spread."""
    def codes(*shape):
        c = torch.randint(0, 256, shape, generator=g, device="cuda").to(torch.uint8)
        return torch.where((c & 0x7F) == 0x7F, c & 0x80, c)
    nkb = -(-K // 128)
    xs = torch.exp2((torch.rand(S, nkb, generator=g, device="cuda") * 2 - 1) * scale_spread)
    ws = torch.exp2((torch.rand(E, -(-N // 128), nkb, generator=g, device="cuda") * 2 - 1) * scale_spread)
    return codes(S, K), xs, codes(E, N, K), ws


def fp8_reference(xq, xs, wq, ws, counts, start):
    S, K = xq.shape
    E, N, _ = wq.shape
    col, row = torch.arange(K) // 128, torch.arange(N) // 128
    x = xq.cpu().view(torch.float8_e4m3fn).double() * xs.cpu().double()[:, col]
    out = torch.zeros(S, N, dtype=torch.float64)
    mag = torch.zeros_like(out)
    r = start
    for e, n in enumerate(counts):
        w = wq[e].cpu().view(torch.float8_e4m3fn).double() * ws[e].cpu().double()[row][:, col]
        out[r:r + n] = x[r:r + n] @ w.T
        mag[r:r + n] = x[r:r + n].abs() @ w.abs().T
        r += n
    return out, mag


@pytest.mark.parametrize("grp", range(len(GROUPS)))
@pytest.mark.parametrize("shape", [(8, 16), (24, 80), (128, 128), (136, 272), (264, 144), (1000, 208), (72, 1168)])
def test_fp8_grouped_matches_64_bit_sums(grp, shape):
    c = GROUPS[grp]
    N, K = shape
    counts, start = c["counts"], c["start"]
    S = start + sum(counts) + c["spare"]
    out_dtype = (torch.bfloat16, torch.float32)[(grp + N // 8) % 2]
    ops = fp8_operands(gen(grp * 1000 + N), S, len(counts), N, K)
    got = B.situ_moe_fp8_grouped_gemm(*ops, offsets_of(counts, start), out_dtype=out_dtype)
    ref, mag = fp8_reference(*ops, counts, start)
    assert_sum(got, ref, mag, K, out_dtype)


@pytest.mark.parametrize("S,N,K", [(1, 8, 16), (1, 512, 1024), (3, 2048, 4096), (16, 136, 7168), (33, 6144, 640),
                                   (70, 264, 1040), (129, 1000, 2064), (700, 1032, 1296), (2000, 264, 144)])
def test_fp8_dense_matches_64_bit_sums(S, N, K):
    xq, xs, wq, ws = fp8_operands(gen(S), S, 1, N, K)
    for out_dtype in (torch.bfloat16, torch.float32):
        got = B.situ_moe_fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=out_dtype)
        ref, mag = fp8_reference(xq, xs, wq, ws, [S], 0)
        assert_sum(got, ref, mag, K, out_dtype)


# wide tiles on one CTA and on pairs, with N's last tile in its first half, at
# its end and in its second half, K's last block partial, and groups that end
# in either CTA's rows; then the narrow forms split over clusters
@pytest.mark.parametrize("counts,N,K", [
    ([75, 0, 128, 129, 40, 90, 3, 200, 110], 2056, 208), ([60, 70, 80, 90, 100, 50, 40, 130], 2048, 1040),
    ([257, 600, 0, 1, 511, 256], 2184, 144), ([640, 128, 700], 2056, 1168), ([900], 1928, 272),
    ([4500, 4000], 264, 128), ([300, 700], 2056, 256),
    ([17], 264, 4112), ([3, 0, 12, 9], 136, 2064), ([64], 264, 3088), ([100, 20], 136, 2192)])
def test_every_form_of_the_fp8_product(counts, N, K):
    S = 2 + sum(counts) + 3
    ops = fp8_operands(gen(N + K), S, len(counts), N, K)
    ref, mag = fp8_reference(*ops, counts, 2)
    for out_dtype in (torch.bfloat16, torch.float32):
        got = B.situ_moe_fp8_grouped_gemm(*ops, offsets_of(counts, 2), out_dtype=out_dtype)
        assert_sum(got, ref, mag, K, out_dtype)


# Wide tiles write whole boxes of 32 rows and, at a group's end, single rows:
# into a part of a larger array, what lies beside it and the rows of no expert
# stay as they were.
@pytest.mark.parametrize("counts,N,K", [
    ([1100, 0, 2501, 33, 1600], 264, 256), ([1025, 31, 4000], 2184, 128),       # pairs, rows on lines
    ([170, 0, 333, 32, 500], 1928, 144), ([900], 72, 1040),                    # pairs, rows off the lines
    ([75, 0, 128, 129, 40, 190, 31], 2056, 256), ([1000, 20, 3, 0, 960], 136, 384)])   # one CTA
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_fp8_wide_tiles_write_their_rows_only(counts, N, K, out_dtype):
    S, start = sum(counts) + 9, 4
    ops = fp8_operands(gen(N + K), S, len(counts), N, K)
    ref, mag = fp8_reference(*ops, counts, start)
    big = torch.full((S + 2, N + 24), 77.0, device="cuda", dtype=out_dtype)
    out = big[1:1 + S, 8:8 + N]
    got = B.situ_moe_fp8_grouped_gemm(*ops, offsets_of(counts, start), out=out, zero_rest=False)
    assert got is out
    end = start + sum(counts)
    assert_sum(out[start:end], ref[start:end], mag[start:end], K, out_dtype)
    assert (out[:start] == 77).all() and (out[end:] == 77).all()
    assert (big[0] == 77).all() and (big[-1] == 77).all() and (big[:, :8] == 77).all() and (big[:, 8 + N:] == 77).all()
    twice = B.situ_moe_fp8_grouped_gemm(*ops, offsets_of(counts, start))
    again = B.situ_moe_fp8_grouped_gemm(*ops, offsets_of(counts, start))
    assert torch.equal(twice, again)


# Weights that are a part of a larger array are read where they lie: the same
# bits as from a copy, and no copy made; what surrounds them is NaN.
@pytest.mark.parametrize("counts,N,K", [([5, 0, 20], 264, 2064), ([90, 60, 0, 97], 1416, 208),
                                        ([300, 700], 2056, 256), ([9000, 0, 10000], 72, 128)])
@pytest.mark.parametrize("part", ["rows", "columns", "both"])
def test_products_read_parts_of_weights_in_place(counts, N, K, part):
    E, S, off = len(counts), sum(counts) + 2, offsets_of(counts, 1)
    r0, c0 = (N if part != "columns" else 0), (16 if part != "rows" else 0)
    shape = (E, r0 + N + (8 if r0 else 0), c0 + K + (32 if c0 else 0))
    g = gen(N + K)
    x = torch.randn(S, K, device="cuda", generator=g).bfloat16()
    dy = torch.randn(S, N, device="cuda", generator=g).bfloat16()
    w = torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16)[:, r0:r0 + N, c0:c0 + K]
    wc = torch.randn(E, N, K, device="cuda", generator=g).bfloat16()
    w.copy_(wc)
    xq, xs, wq, ws = fp8_operands(g, S, E, N, K)
    wv = torch.full(shape, 127, device="cuda", dtype=torch.uint8)[:, r0:r0 + N, c0:c0 + K]   # E4M3 NaN
    wv.copy_(wq)
    assert not w.is_contiguous() and not wv.is_contiguous()
    for make, small in ((lambda v: B.situ_moe_grouped_gemm(x, v, off), (w, wc)),
                        (lambda v: B.situ_moe_grouped_gemm_dgrad(dy, v, off, out_dtype=torch.float32), (w, wc)),
                        (lambda v: B.situ_moe_fp8_grouped_gemm(xq, xs, v, ws, off), (wv, wq))):
        ref = make(small[1])
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_stats()["requested_bytes.all.current"]
        got = make(small[0])
        torch.cuda.synchronize()
        grown = torch.cuda.memory_stats()["requested_bytes.all.peak"] - before
        assert grown <= got.numel() * got.element_size()
        assert torch.isfinite(got).all() and torch.equal(got, ref)
    # one expert's part, and one expert's weights for all (copied)
    y = B.situ_moe_fp8_gemm(xq, xs, wv[0], ws[0])
    assert torch.equal(y, B.situ_moe_fp8_gemm(xq, xs, wq[0], ws[0]))
    one = w[:1].expand(E, N, K)
    assert torch.equal(B.situ_moe_grouped_gemm(x, one, off), B.situ_moe_grouped_gemm(x, one.contiguous(), off))


@pytest.mark.parametrize("counts,N,K", [
    ([(7 * i) % 90 for i in range(40)], 520, 1040),      # 64-token tiles, several a CTA, some groups of two tiles
    ([33] * 45, 640, 128),                               # one block of scales
    ([(5 * i) % 38 for i in range(170)], 136, 1680),     # 32-token tiles, a partial block of rows and of columns
])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_fp8_several_narrow_tiles_per_cta(counts, N, K, out_dtype):
    S = sum(counts) + 6
    ops = fp8_operands(gen(N + K), S, len(counts), N, K)
    ref, mag = fp8_reference(*ops, counts, 3)
    got = B.situ_moe_fp8_grouped_gemm(*ops, offsets_of(counts, 3), out_dtype=out_dtype)
    assert_sum(got, ref, mag, K, out_dtype)


def test_fp8_nan_and_infinite_scales_stay_in_their_rows():
    # wide tiles: a NaN code in one row, an infinite scale in another, and rows
    # of no group full of NaN, leave every other row alone
    counts, N, K = [300, 0, 400, 350], 2056, 400
    S = 4 + sum(counts) + 2
    xq, xs, wq, ws = fp8_operands(gen(44), S, 4, N, K)
    xq[:4] = 0x7F
    xs[-2:] = float("nan")
    xq[4 + 299, 7] = 0x7F
    xs[4 + 300, 1] = float("inf")
    y = B.situ_moe_fp8_grouped_gemm(xq, xs, wq, ws, offsets_of(counts, 4), out_dtype=torch.float32)
    xq[4 + 299, 7], xs[4 + 300, 1] = 0, 1.0
    ref, mag = fp8_reference(xq[4:-2], xs[4:-2], wq, ws, counts, 0)
    assert (y[:4] == 0).all() and (y[-2:] == 0).all()
    assert y[4 + 299].isnan().all() and not y[4 + 300].isfinite().any()
    keep = torch.ones(sum(counts), dtype=torch.bool)
    keep[299:301] = False
    assert_sum(y[4:-2][keep.cuda()], ref[keep], mag[keep], K, torch.float32)


def test_fp8_bad_offsets_stay_inside_the_operands():
    for S, N, K in ((50, 64, 64), (900, 2056, 144)):
        xq, xs, wq, ws = fp8_operands(gen(45), S, 4, N, K)
        off = torch.tensor([0, 10, 5, 2000000000, 60], dtype=torch.int32, device="cuda")
        y = B.situ_moe_fp8_grouped_gemm(xq, xs, wq, ws, off)
        assert y.shape == (S, N) and B.situ_moe_gemm_status() == 0


def test_fp8_split_repeats_bits_and_other_streams():
    xq, xs, wq, ws = fp8_operands(gen(46), 9, 1, 264, 4112)
    y1 = B.situ_moe_fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = B.situ_moe_fp8_gemm(xq, xs, wq[0], ws[0], out_dtype=torch.float32, stream=s)
    # a layout that is copied first: the copy belongs to that stream as well
    wide = torch.zeros(9, 4112 + 48, dtype=torch.uint8, device="cuda")
    wide[:, 5:5 + 4112] = xq
    s.wait_stream(torch.cuda.current_stream())
    y3 = B.situ_moe_fp8_gemm(wide[:, 5:5 + 4112], xs, wq[0], ws[0], out_dtype=torch.float32, stream=s)
    q, sc = B.situ_moe_quant_fp8(y1, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and torch.equal(y1, y3)
    q2, sc2 = B.situ_moe_quant_fp8(y1)
    assert torch.equal(q, q2) and torch.equal(sc, sc2)


def test_fp8_rows_of_no_expert_and_other_groups():
    counts, N, K = [40, 1, 0, 70], 264, 400
    S = 2 + sum(counts) + 5
    xq, xs, wq, ws = fp8_operands(gen(41), S, 4, N, K)
    off = offsets_of(counts, 2)
    xq[:2] = 0x7F                      # NaN rows of no expert
    xs[-5:] = float("inf")
    wq[1] = 0x7F                       # one expert's weights are NaN
    out = torch.full((S, N + 8), 3.0, device="cuda")
    y = B.situ_moe_fp8_grouped_gemm(xq, xs, wq, ws, off, out=out[:, :N])
    ref, mag = fp8_reference(xq[2:-5], xs[2:-5], wq, ws, counts, 0)
    assert (y[:2] == 0).all() and (y[-5:] == 0).all() and y[42].isnan().all() and (out[:, N:] == 3).all()
    keep = torch.arange(sum(counts)) != 40
    assert_sum(y[2:-5][keep.cuda()], ref[keep], mag[keep], K, torch.float32)
    kept = torch.full((S, N), 3.0, device="cuda")
    B.situ_moe_fp8_grouped_gemm(xq, xs, wq, ws, off, out=kept, zero_rest=False)
    assert (kept[:2] == 3).all() and (kept[-5:] == 3).all()


def test_fp8_strided_rows_and_float8_dtype():
    S, N, K = 20, 64, 256
    xq, xs, wq, ws = fp8_operands(gen(42), S, 1, N, K)
    ref, mag = fp8_reference(xq, xs, wq, ws, [S], 0)
    wide = torch.zeros(S, K + 48, dtype=torch.uint8, device="cuda")
    for at in (16, 5):                 # in place, and misaligned: copied
        wide[:, at:at + K] = xq
        got = B.situ_moe_fp8_gemm(wide[:, at:at + K], xs, wq[0], ws[0], out_dtype=torch.float32)
        assert_sum(got, ref, mag, K, torch.float32)
    got = B.situ_moe_fp8_gemm(xq.view(torch.float8_e4m3fn), xs.T.contiguous().T, wq[0].view(torch.float8_e4m3fn), ws[0],
                              out_dtype=torch.float32)
    assert_sum(got, ref, mag, K, torch.float32)


def test_quantised_product_is_near_the_unquantised():
    # E4M3 keeps 4 significant bits: 2^-4 relative per factor, so 2^-3 of the
    # magnitudes' sum bounds the quantised product's distance
    S, N, K = 50, 264, 1040
    g = gen(43)
    x, w = normal(g, S, K), normal(g, N, K, std=0.05)
    y = B.situ_moe_fp8_gemm(*B.situ_moe_quant_fp8(x), *B.situ_moe_quant_fp8(w, 128), out_dtype=torch.float32)
    ref = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    assert ((y.double() - ref).abs() <= 2.0 ** -3 * mag).all()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_python_refusals():
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    off = offsets_of([2, 2])
    with pytest.raises(TypeError):
        B.situ_moe_grouped_gemm(x.half(), w, off)                       # mixed types
    with pytest.raises(TypeError):
        B.situ_moe_grouped_gemm(x.float(), w.float(), off)
    with pytest.raises(TypeError):
        B.situ_moe_grouped_gemm(x, w, off.long())
    with pytest.raises(TypeError):
        B.situ_moe_grouped_gemm(x, w, off, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm(x, w, off[:2])                          # one group, two experts
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm(x[:, :32], w, off)
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm(x.cpu(), w.cpu(), off.cpu())
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm(x, w, off.cpu())
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm(x, w, off, out=torch.zeros(4, 63, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm(x, w, off, out=torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").T)
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm_wgrad(x, x, off, accumulate=True)
    with pytest.raises(B.SituError) as e:
        B.situ_moe_grouped_gemm(x[:, :60].contiguous(), w[:, :, :60].contiguous(), off)   # K not a multiple of 8
    assert e.value.status == 2
    q, s = torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, device="cuda")
    wq, ws = torch.zeros(64, 64, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, device="cuda")
    with pytest.raises(TypeError):
        B.situ_moe_fp8_gemm(q.float(), s, wq, ws)
    with pytest.raises(TypeError):
        B.situ_moe_fp8_gemm(q, s, wq, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        B.situ_moe_fp8_gemm(q, s[:3], wq, ws)
    with pytest.raises(ValueError):
        B.situ_moe_fp8_gemm(q, s, wq, ws.reshape(1, 1, 1))
    with pytest.raises(B.SituError) as e:
        B.situ_moe_fp8_gemm(q[:, :56].contiguous(), s, wq[:, :56].contiguous(), ws)       # K not a multiple of 16
    assert e.value.status == 2
    with pytest.raises(ValueError):
        B.situ_moe_quant_fp8(x, 64)
    with pytest.raises(TypeError):
        B.situ_moe_quant_fp8(x.double())
    torch.cuda.synchronize()


def test_a_given_up_wait_stops_later_products():
    # the status word as a kernel that gave up leaves it: no work until reset
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, 64, 64, dtype=torch.bfloat16, device="cuda")
    off = offsets_of([4])
    B._status_word(x.device.index).fill_(74)
    out = torch.full((4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    B.situ_moe_grouped_gemm(x, w, off, out=out)
    assert (out == 5).all()
    assert B.situ_moe_gemm_status(reset=True) == 74
    B.situ_moe_grouped_gemm(x, w, off, out=out)
    assert (out == 64).all() and B.situ_moe_gemm_status() == 0
