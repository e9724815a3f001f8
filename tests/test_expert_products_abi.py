"""Host-side checks of the expert products' entry points (no GPU needed): bad
arguments are refused before anything is launched."""
import ctypes

import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def grouped(lib, **over):
    a = dict(direction=0, dtype=0, out_dtype=0, S=16, N=64, K=128, E=4, accumulate=0, keep_rest=0, a=0x1000, lda=128,
             b=0x2000, ldb=128, offsets=0x3000, out=0x4000, ldo=64, device_status=0x5000)
    a.update(over)
    return lib.situ_moe_grouped_gemm(ctypes.byref(B.SituGroupedGemmArgs(**a)), None)


@pytest.mark.parametrize("over,status", [
    (dict(direction=3), 3), (dict(direction=-1), 3), (dict(dtype=2), 3), (dict(dtype=1), 3), (dict(out_dtype=1), 3),
    (dict(out_dtype=7), 3), (dict(accumulate=1), 3), (dict(accumulate=2, direction=2), 3), (dict(keep_rest=2), 3),
    (dict(keep_rest=1, direction=2), 3),
    (dict(S=-1), 2), (dict(N=0), 2), (dict(N=60), 2), (dict(K=4), 2), (dict(K=132), 2), (dict(E=0), 2),
    (dict(E=1025), 2), (dict(K=1 << 21), 2), (dict(lda=120), 2), (dict(lda=132), 2), (dict(ldo=56), 2),
    (dict(ldo=68), 2), (dict(direction=1, lda=56), 2), (dict(direction=1, ldo=120), 2),
    (dict(direction=2, lda=64, ldb=120), 2), (dict(direction=2, lda=56), 2),
    (dict(a=None), 1), (dict(b=None), 1), (dict(offsets=None), 1), (dict(out=None), 1), (dict(device_status=None), 1),
    (dict(a=0x1008), 6), (dict(b=0x2008), 6), (dict(out=0x4008), 6), (dict(offsets=0x3002), 6),
    (dict(device_status=0x5001), 6),
    (dict(S=0, a=None, b=None), 0),          # nothing to do, nothing launched
    (dict(S=0, direction=2, accumulate=1, lda=64), 0),
])
def test_grouped_refusals(lib, over, status):
    assert grouped(lib, **over) == status


def fp8(lib, **over):
    a = dict(out_dtype=0, S=16, N=64, K=128, E=1, keep_rest=0, x_q=0x1000, ldx=128, x_scale=0x2000, w_q=0x3000,
             w_scale=0x4000, offsets=None, out=0x5000, ldo=64, device_status=0x6000)
    a.update(over)
    return lib.situ_moe_fp8_gemm(ctypes.byref(B.SituFp8GemmArgs(**a)), None)


@pytest.mark.parametrize("over,status", [
    (dict(out_dtype=1), 3), (dict(keep_rest=3), 3),
    (dict(S=-1), 2), (dict(N=4), 2), (dict(N=60), 2), (dict(K=8), 2), (dict(K=136), 2), (dict(E=2), 2),
    (dict(E=1025, offsets=0x7000), 2), (dict(ldx=112), 2), (dict(ldx=136), 2), (dict(ldo=56), 2), (dict(ldo=68), 2),
    (dict(x_q=None), 1), (dict(x_scale=None), 1), (dict(w_q=None), 1), (dict(w_scale=None), 1), (dict(out=None), 1),
    (dict(device_status=None), 1),
    (dict(x_q=0x1008), 6), (dict(w_q=0x3008), 6), (dict(out=0x5008), 6), (dict(x_scale=0x2002), 6),
    (dict(w_scale=0x4001), 6), (dict(offsets=0x7001), 6), (dict(device_status=0x6002), 6),
    (dict(S=0, x_q=None), 0),
])
def test_fp8_refusals(lib, over, status):
    assert fp8(lib, **over) == status


@pytest.mark.parametrize("args,status", [
    ((0x1000, 3, 1, 4, 128, 128, 1, 0x2000, 0x3000), 3), ((0x1000, 0, 1, 4, 128, 128, 64, 0x2000, 0x3000), 3),
    ((0x1000, 0, 1, 4, 12, 16, 1, 0x2000, 0x3000), 2), ((0x1000, 0, 1, 4, 128, 120, 1, 0x2000, 0x3000), 2),
    ((0x1000, 0, 1, 4, 128, 132, 1, 0x2000, 0x3000), 2), ((0x1000, 0, 1, -1, 128, 128, 1, 0x2000, 0x3000), 2),
    ((None, 0, 1, 4, 128, 128, 1, 0x2000, 0x3000), 1), ((0x1000, 0, 1, 4, 128, 128, 1, None, 0x3000), 1),
    ((0x1000, 0, 1, 4, 128, 128, 1, 0x2000, None), 1), ((0x1008, 0, 1, 4, 128, 128, 1, 0x2000, 0x3000), 6),
    ((0x1000, 0, 1, 4, 128, 128, 1, 0x2004, 0x3000), 6), ((0x1000, 0, 1, 4, 128, 128, 1, 0x2000, 0x3002), 6),
    ((None, 0, 1, 0, 128, 128, 1, None, None), 0), ((None, 0, 0, 4, 128, 128, 128, None, None), 0),
])
def test_quant_refusals(lib, args, status):
    assert lib.situ_moe_quant_fp8(*args, None) == status


@pytest.mark.parametrize("over,status", [
    (dict(ldw=120), 2), (dict(ldw=132), 2), (dict(ldw=-128), 2), (dict(ldw=1 << 62), 2),
    (dict(stride_w=63 * 128), 2), (dict(stride_w=64 * 128 + 8), 2), (dict(ldw=256, stride_w=64 * 128), 2),
    (dict(stride_w=-64 * 128), 2), (dict(direction=2, lda=64, ldw=128), 2), (dict(direction=2, lda=64, stride_w=64 * 128), 2),
    (dict(S=0, ldw=256), 0), (dict(S=0, ldw=256, stride_w=128 * 256), 0),
])
def test_grouped_refuses_weight_strides(lib, over, status):
    assert grouped(lib, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(ldw=112), 2), (dict(ldw=136), 2), (dict(ldw=1 << 62), 2), (dict(stride_w=64 * 112), 2),
    (dict(ldw=256, stride_w=64 * 256 + 128), 2), (dict(S=0, ldw=144, stride_w=65 * 144), 0),
])
def test_fp8_refuses_weight_strides(lib, over, status):
    assert fp8(lib, **over) == status


def test_null_args(lib):
    assert lib.situ_moe_grouped_gemm(None, None) == 1
    assert lib.situ_moe_fp8_gemm(None, None) == 1


def test_binding_refuses_host_tensors():
    w, off = torch.zeros(1, 64, 64, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (B.situ_moe_grouped_gemm, B.situ_moe_grouped_gemm_dgrad):
        with pytest.raises(ValueError):
            f(x, w, off)
    with pytest.raises(ValueError):
        B.situ_moe_grouped_gemm_wgrad(x, x, off)
    with pytest.raises(ValueError):
        B.situ_moe_quant_fp8(x)
