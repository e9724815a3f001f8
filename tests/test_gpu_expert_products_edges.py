"""Edges of the expert products on the GPU: sequences of tiles, offsets, sizes
and values at which an operator could go wrong without its ordinary cases
showing it.  Bars as in test_gpu_expert_products.py; most comparisons are bit
for bit.
"""
import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build
from test_gpu_expert_products import HALF_ULP, call, fp8_operands, gen, normal, offsets_of, operands, plain_quant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()
    yield
    assert B.situ_moe_gemm_status() == 0


# Pairs with two output boxes per warp, in sequences where a warp goes from a
# whole tile to a group's end and back.  One block of K leaves the least time
# between a box's uses.  Weights off the 128-byte lines take the form with one
# box, whose sums are the same.
@pytest.mark.parametrize("counts,N", [([8200], 6144), ([2000] * 8, 2048), ([1025, 4033, 1100, 3], 2184)])
@pytest.mark.parametrize("K", [128, 256])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_fp8_output_boxes_in_turn(counts, N, K, out_dtype):
    S, E = sum(counts), len(counts)
    xq, xs, wq, ws = fp8_operands(gen(N + K), S, E, N, K)
    off = offsets_of(counts)
    apart = torch.zeros(E, N, K + 16, dtype=torch.uint8, device="cuda")[:, :, :K]
    apart.copy_(wq)
    want = B.situ_moe_fp8_grouped_gemm(xq, xs, apart, ws, off, out_dtype=out_dtype)
    assert torch.isfinite(want).all()
    for _ in range(8):
        assert torch.equal(B.situ_moe_fp8_grouped_gemm(xq, xs, wq, ws, off, out_dtype=out_dtype), want)


# Offsets that descend or leave [0, S] are clamped to ascending order: the
# results are those of the clamped array, and the same on every call.  Groups
# taken pair by pair would overlap here, with more tiles than a split launch
# (few tiles) has clusters.
BAD_OFFSETS = [[0, 10, 5, 2000000000, 60], [50, 0, 50, 0, 50, 0, 50], [-7, -2147483648, 3, 2, 9], [40, 30, 20, 10],
               [0, 1 << 30, 0, 2147483647, -1]]


@pytest.mark.parametrize("bad", BAD_OFFSETS + [[(37 * i) % 1200 - 100 for i in range(1025)]])
@pytest.mark.parametrize("S,N,K", [(50, 264, 2064), (900, 136, 144), (1500, 2056, 128)])
def test_offsets_are_clamped_to_ascending_order(bad, S, N, K):
    E = len(bad) - 1
    if E > 100:
        N = 136
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    ok = torch.cummax(off.clamp(0, S), 0).values.int()
    g = gen(S + E)
    x, dy, w = normal(g, S, K), normal(g, S, N), normal(g, E, N, K, std=0.1)
    fp8 = fp8_operands(g, S, E, N, K)
    for out_dtype in (torch.bfloat16, torch.float32):
        for f in (lambda o: B.situ_moe_grouped_gemm(x, w, o, out_dtype=out_dtype),
                  lambda o: B.situ_moe_grouped_gemm_dgrad(dy, w, o, out_dtype=out_dtype),
                  lambda o: B.situ_moe_grouped_gemm_wgrad(dy, x, o, out_dtype=out_dtype),
                  lambda o: B.situ_moe_fp8_grouped_gemm(*fp8, o, out_dtype=out_dtype)):
            want = f(ok)
            assert torch.isfinite(want).all()
            for _ in range(3):
                assert torch.equal(f(off), want)


# The codes are compared as bytes: zeros, and values that round to zero, keep
# their sign, in blocks whose scale the fast quotient takes and in others.
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("amax", [0.0, 1e-7, 1.0, 3000.0, 1e-37, 1e30])
def test_quant_keeps_the_sign_of_zero(rows, dtype, amax):
    g = gen(int(rows + amax % 97))
    x = torch.randint(-4, 5, (2 * rows + 3, 264), generator=g, device="cuda").float() * (amax / 4)
    x[:, 1::3] = -0.0
    x[:, 2::9] *= 1e-5                  # rounds to a zero of either sign
    x = x.to(dtype)
    if dtype == torch.float16 and not torch.isfinite(x).all():
        pytest.skip("beyond f16")
    q, s = B.situ_moe_quant_fp8(x, rows)
    rq, rs = plain_quant(x, rows)
    assert torch.equal(s.cpu(), rs)
    assert (rq.view(torch.uint8) == 0x80).any()
    assert torch.equal(q.cpu(), rq.view(torch.uint8))


# Long contractions with terms of one sign, where truncated additions would
# pile up.  The bar: the rounding to 16 bits, 2^-23 per element of a chunk of
# 512 that the tensor cores add, and 2^-24 per rounded addition of a chunk.
def long_bar(ref, L, dtype):
    return ref * ((512 * 2.0 ** -23 + -(-L // 512) * 2.0 ** -24) * (1 + HALF_ULP[dtype]) + HALF_ULP[dtype])


@pytest.mark.parametrize("dtype,log2", [(torch.float16, 14), (torch.float16, 18), (torch.bfloat16, 17), (torch.bfloat16, 19)])
def test_long_weight_gradients_of_one_sign(dtype, log2):
    N, K, S = 1024, 2560, 1 << log2
    g = gen(log2)
    dy = (torch.rand(S, N, generator=g, device="cuda") * 2.0 ** (12 - log2)).to(dtype)
    x = torch.rand(S, K, generator=g, device="cuda").to(dtype)
    got = B.situ_moe_grouped_gemm_wgrad(dy, x, offsets_of([S]))[0, :48].double()
    ref = sum(dy[i:i + 65536, :48].double().T @ x[i:i + 65536].double() for i in range(0, S, 65536))
    assert ((got - ref).abs() <= long_bar(ref, S, dtype)).all()


@pytest.mark.parametrize("direction", ["forward", "dgrad"])
@pytest.mark.parametrize("dtype,log2", [(torch.float16, 17), (torch.bfloat16, 18)])
def test_long_products_of_one_sign(direction, dtype, log2):
    M, L, S = 4096, 1 << log2, 300
    g = gen(log2)
    a = (torch.rand(S, L, generator=g, device="cuda") * 2.0 ** (12 - log2)).to(dtype)
    w = torch.rand(1, *((M, L) if direction == "forward" else (L, M)), generator=g, device="cuda", dtype=torch.float16).to(dtype)
    got = call(direction, a, w, offsets_of([S]))[:, :48].double()
    part = w[0, :48].T if direction == "forward" else w[0][:, :48]
    ref = a.double() @ part.double()
    assert ((got - ref).abs() <= long_bar(ref, L, dtype)).all()


# the 16-bit results of long contractions in every form of tile: groups short,
# empty and uneven, sizes off the tiles
@pytest.mark.parametrize("counts,M", [([(7 * i) % 24 for i in range(160)], 136), ([(11 * i) % 60 for i in range(60)], 264),
                                      ([70, 90, 0, 97, 5] * 8, 520), ([20000], 120), ([300, 0, 700, 129, 1], 2312)])
@pytest.mark.parametrize("direction", ["forward", "dgrad"])
def test_long_products_in_every_form(counts, M, direction):
    L, S, E = 8200, sum(counts) + 5, len(counts)
    N, K = (M, L) if direction == "forward" else (L, M)
    a, b, _ = operands(direction, gen(M), S, E, N, K, torch.float16)
    off = offsets_of(counts, 2)
    got = call(direction, a, b, off)
    want = call(direction, a, b, off, out_dtype=torch.float32)     # the same sums, rounded once
    assert torch.isfinite(want).all() and (want != 0).any()
    assert torch.equal(got, want.half())


@pytest.mark.parametrize("counts,N,K", [([9000, 0, 37, 5], 1000, 2056), ([8200], 120, 20488), ([16, 8300, 33, 64, 65], 264, 5000)])
def test_long_weight_gradients_in_every_form(counts, N, K):
    S = sum(counts) + 5
    dy, x, _ = operands("wgrad", gen(N), S, len(counts), N, K, torch.float16)
    off = offsets_of(counts, 2)
    got = B.situ_moe_grouped_gemm_wgrad(dy, x, off)
    want = B.situ_moe_grouped_gemm_wgrad(dy, x, off, out_dtype=torch.float32)
    assert torch.isfinite(want).all() and torch.equal(got, want.half())


def test_operands_of_another_stream_outlive_their_last_reference():
    # the side stream is held up while the operands are dropped: their memory
    # must not come back for anyone else until its work is done
    counts, N, K = [40, 0, 25], 136, 272
    S = sum(counts)
    g = gen(71)
    off = offsets_of(counts)
    big = normal(g, S, 1 << 16)                      # a block of its own size
    x, w, dy = normal(g, S, K), normal(g, 3, N, K, std=0.1), normal(g, S, N)
    fp8 = fp8_operands(g, S, 3, N, K)
    calls = {
        "forward": (B.situ_moe_grouped_gemm, (x, w, off)), "dgrad": (B.situ_moe_grouped_gemm_dgrad, (dy, w, off)),
        "wgrad": (B.situ_moe_grouped_gemm_wgrad, (dy, x, off)), "quant": (B.situ_moe_quant_fp8, (big,)),
        "fp8": (B.situ_moe_fp8_grouped_gemm, (*fp8, off)),
        "dense": (B.situ_moe_fp8_gemm, (fp8[0], fp8[1], fp8[2][0].clone(), fp8[3][0].clone())),
    }
    side = torch.cuda.Stream()
    for name, (f, operands_) in calls.items():
        want = f(*operands_)
        mine = [t.clone() for t in operands_]
        at = {t.data_ptr() for t in mine}
        shapes = [(t.shape, t.dtype) for t in mine]
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)           # about 50 ms
        got = f(*mine, stream=side)
        del mine
        others = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(4)]
        assert not at & {t.data_ptr() for t in others}, name
        torch.cuda.synchronize()
        got, want = (got, want) if isinstance(got, tuple) else ((got,), (want,))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_a_given_result_of_another_stream_outlives_its_last_reference():
    x, w, off = torch.ones(40, 64, device="cuda").bfloat16(), torch.ones(1, 64, 64, device="cuda").bfloat16(), offsets_of([40])
    side = torch.cuda.Stream()
    out, q, s = torch.empty(40, 64, device="cuda"), torch.empty(40, 64, dtype=torch.uint8, device="cuda"), torch.empty(40, 1, device="cuda")
    at = {t.data_ptr() for t in (out, q, s)}
    shapes = [(t.shape, t.dtype) for t in (out, q, s)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    B.situ_moe_grouped_gemm(x, w, off, out=out, stream=side)
    B.situ_moe_quant_fp8(x, out=(q, s), stream=side)
    del out, q, s
    others = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(4)]
    assert not at & {t.data_ptr() for t in others}
    torch.cuda.synchronize()
