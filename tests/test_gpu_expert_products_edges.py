"""Edges of the expert products on the GPU: sequences of tiles, offsets, sizes
and values at which an operator could go wrong without its ordinary cases
showing it.  Bars as in test_gpu_expert_products.py; most comparisons are bit
for bit.
"""
import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build
from test_gpu_expert_products import fp8_operands, gen, offsets_of

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
