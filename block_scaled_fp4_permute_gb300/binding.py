"""ctypes binding of ``libsitu_moe.so`` (C ABI in ``include/situ_moe.h``).

Argument marshalling only: PyTorch provides device memory and the stream,
every step of the layer runs in the library's CUDA kernels.  There is no
fallback: if the library is not built, or a call returns an error status,
the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

import torch

from . import build as _build

SITU_OK = 0
SITU_ERR_DEVICE_TIMEOUT = 7
SITU_ACT_BF16, SITU_ACT_MXFP8, SITU_ACT_NVFP4 = 0, 1, 2
SITU_ACT_FN_SITU, SITU_ACT_FN_SWIGLU_BIAS = 0, 1
SITU_W_MXFP4, SITU_W_NVFP4 = 0, 1

SITU_DT_BF16, SITU_DT_F16, SITU_DT_F32 = 0, 1, 2
SITU_GROUPED_FORWARD, SITU_GROUPED_DGRAD, SITU_GROUPED_WGRAD = 0, 1, 2

_lib = None
_lock = threading.Lock()


class SituError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


class SituMoeArgs(ctypes.Structure):
    """Mirror of ``situ_moe_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "T", "H", "I", "num_experts_total", "num_local_experts", "local_expert_offset", "top_k",
        "act_dtype", "weight_dtype")] + [(n, ctypes.c_void_p) for n in (
            "hidden_states", "hidden_states_q", "hidden_states_scale", "hidden_states_gscale",
            "topk_ids", "topk_weights", "w1", "w1_scale", "w1_gscale", "w2", "w2_scale",
            "w2_gscale", "gemm1_alpha", "gemm1_beta", "g1_alphas", "g1_alphas_up", "g2_alphas",
            "out", "scales_packed")] + [(n, ctypes.c_int32) for n in (
                "fuse_combine", "activation", "apply_topk_in_fc1", "h1_nvfp4")] + [("tactic", ctypes.c_int32 * 2)]


class SituGroupedGemmArgs(ctypes.Structure):
    """Mirror of ``situ_grouped_gemm_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("direction", "dtype", "out_dtype", "S", "N", "K", "E", "accumulate",
                                              "keep_rest")] + [
        ("a", ctypes.c_void_p), ("lda", ctypes.c_int64), ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64),
        ("offsets", ctypes.c_void_p), ("out", ctypes.c_void_p), ("ldo", ctypes.c_int64),
        ("device_status", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("stride_w", ctypes.c_int64)]


class SituFp8GemmArgs(ctypes.Structure):
    """Mirror of ``situ_fp8_gemm_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("out_dtype", "S", "N", "K", "E", "keep_rest")] + [
        ("x_q", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_scale", ctypes.c_void_p), ("w_q", ctypes.c_void_p),
        ("w_scale", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("ldo", ctypes.c_int64), ("device_status", ctypes.c_void_p), ("ldw", ctypes.c_int64),
        ("stride_w", ctypes.c_int64)]


class SituBalanceArgs(ctypes.Structure):
    """Mirror of ``situ_balance_args``."""
    _fields_ = [("router_logits", ctypes.c_void_p), ("ld", ctypes.c_int64), ("topk_ids", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("T", ctypes.c_int32), ("num_experts_total", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("coef", ctypes.c_float), ("loss", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("row_stats", ctypes.c_void_p)]


class SituRouterBackwardArgs(ctypes.Structure):
    """Mirror of ``situ_router_backward_args``."""
    _fields_ = [("router_logits", ctypes.c_void_p), ("ld", ctypes.c_int64), ("topk_ids", ctypes.c_void_p),
                ("mask", ctypes.c_void_p)] + [(n, ctypes.c_int32) for n in (
                    "T", "num_experts_total", "top_k", "renormalize")] + [("coef", ctypes.c_float)] + [
        (n, ctypes.c_void_p) for n in ("counts", "tokens", "row_stats", "dloss", "topk_weights", "dweights", "dlogits")] + [
        ("ldo", ctypes.c_int64)]


class SituGatedArgs(ctypes.Structure):
    """Mirror of ``situ_gated_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "activation", "S", "I", "E")] + [
        ("gate_up", ctypes.c_void_p), ("ld_gate_up", ctypes.c_int64), ("p0", ctypes.c_void_p), ("p1", ctypes.c_void_p),
        ("offsets", ctypes.c_void_p), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("q", ctypes.c_void_p),
        ("scale", ctypes.c_void_p), ("dh", ctypes.c_void_p), ("ld_dh", ctypes.c_int64), ("dgate_up", ctypes.c_void_p),
        ("ld_dgate_up", ctypes.c_int64)]


class SituLoraArgs(ctypes.Structure):
    """Mirror of ``situ_lora_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "out_dtype", "S", "K", "N", "r", "n")] + [
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
        ("ids", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("base", ctypes.c_void_p),
        ("ld_base", ctypes.c_int64), ("out", ctypes.c_void_p), ("ldo", ctypes.c_int64), ("u", ctypes.c_void_p),
        ("device_status", ctypes.c_void_p)]


class SituLoraBackwardArgs(ctypes.Structure):
    """Mirror of ``situ_lora_backward_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "dx_dtype", "S", "K", "N", "r", "n")] + [
        ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("u", ctypes.c_void_p), ("dx0", ctypes.c_void_p), ("ld_dx0", ctypes.c_int64), ("dx", ctypes.c_void_p),
        ("ld_dx", ctypes.c_int64), ("da", ctypes.c_void_p), ("db", ctypes.c_void_p), ("device_status", ctypes.c_void_p),
        ("dy_scale", ctypes.c_void_p)]


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise ImportError(f"{path} is missing: build it with "
                                  "`python -m block_scaled_fp4_permute_gb300.build` "
                                  "(the layer has no CPU fallback)")
            l = ctypes.CDLL(path)
            vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            l.situ_status_string.restype = ctypes.c_char_p
            l.situ_status_string.argtypes = [ctypes.c_int]
            l.situ_moe_permute_workspace_size.restype = sz
            l.situ_moe_permute_workspace_size.argtypes = [i32, i32, i32]
            l.situ_moe_permute.restype = ctypes.c_int
            l.situ_moe_permute.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
            l.situ_moe_permute_noalloc.restype = ctypes.c_int
            l.situ_moe_permute_noalloc.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp]
            l.situ_moe_route_topk.restype = ctypes.c_int
            l.situ_moe_route_topk.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
            l.situ_moe_quant_mxfp8.restype = ctypes.c_int
            l.situ_moe_quant_mxfp8.argtypes = [vp, i32, i32, vp, vp, vp]
            l.situ_moe_quant_nvfp4.restype = ctypes.c_int
            l.situ_moe_quant_nvfp4.argtypes = [vp, i32, i32, vp, vp, vp, vp]
            l.situ_moe_workspace_size.restype = sz
            l.situ_moe_workspace_size.argtypes = [ctypes.POINTER(SituMoeArgs)]
            l.situ_moe_forward.restype = ctypes.c_int
            l.situ_moe_forward.argtypes = [ctypes.POINTER(SituMoeArgs), vp, sz, vp]
            l.situ_moe_forward_profiled.restype = ctypes.c_int
            l.situ_moe_forward_profiled.argtypes = [ctypes.POINTER(SituMoeArgs), vp, sz, vp,
                                                    ctypes.POINTER(ctypes.c_void_p)]
            l.situ_moe_packed_scales_size.restype = sz
            l.situ_moe_packed_scales_size.argtypes = [ctypes.POINTER(SituMoeArgs)]
            l.situ_moe_pack_scales.restype = ctypes.c_int
            l.situ_moe_pack_scales.argtypes = [ctypes.POINTER(SituMoeArgs), vp, sz, vp]
            l.situ_moe_forward_launches.restype = ctypes.c_int32
            l.situ_moe_forward_launches.argtypes = [ctypes.POINTER(SituMoeArgs)]
            l.situ_moe_device_status.restype = ctypes.c_int
            l.situ_moe_device_status.argtypes = [ctypes.POINTER(SituMoeArgs), vp, vp,
                                                 ctypes.POINTER(ctypes.c_int32)]
            l.situ_moe_wait_selftest.restype = ctypes.c_int
            l.situ_moe_wait_selftest.argtypes = [vp, vp]
            l.situ_moe_forward_wait_test.restype = ctypes.c_int
            l.situ_moe_forward_wait_test.argtypes = [ctypes.POINTER(SituMoeArgs), vp, sz, vp, i32, i32]
            l.situ_tc_peak.restype = ctypes.c_int
            l.situ_tc_peak.argtypes = [i32, i32, vp, ctypes.POINTER(ctypes.c_double), vp]
            l.situ_moe_grouped_gemm.restype = ctypes.c_int
            l.situ_moe_grouped_gemm.argtypes = [ctypes.POINTER(SituGroupedGemmArgs), vp]
            l.situ_moe_quant_fp8.restype = ctypes.c_int
            l.situ_moe_quant_fp8.argtypes = [vp, i32, i32, i32, i32, ctypes.c_int64, i32, vp, vp, vp]
            l.situ_moe_fp8_gemm.restype = ctypes.c_int
            l.situ_moe_fp8_gemm.argtypes = [ctypes.POINTER(SituFp8GemmArgs), vp]
            i64 = ctypes.c_int64
            l.situ_moe_balance_loss_workspace_size.restype = sz
            l.situ_moe_balance_loss_workspace_size.argtypes = [i32, i32]
            l.situ_moe_balance_loss.restype = ctypes.c_int
            l.situ_moe_balance_loss.argtypes = [ctypes.POINTER(SituBalanceArgs), vp, sz, vp]
            l.situ_moe_router_backward.restype = ctypes.c_int
            l.situ_moe_router_backward.argtypes = [ctypes.POINTER(SituRouterBackwardArgs), vp]
            l.situ_moe_save_mxfp8.restype = ctypes.c_int
            l.situ_moe_save_mxfp8.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp]
            l.situ_moe_restore_mxfp8.restype = ctypes.c_int
            l.situ_moe_restore_mxfp8.argtypes = [vp, vp, i32, i32, i32, vp, i64, vp]
            for fn in (l.situ_moe_gated, l.situ_moe_gated_backward):
                fn.restype = ctypes.c_int
                fn.argtypes = [ctypes.POINTER(SituGatedArgs), vp]
            l.situ_moe_lora_workspace_size.restype = sz
            l.situ_moe_lora_workspace_size.argtypes = [i32, i32, i32, i32, i32]
            l.situ_moe_lora_backward_workspace_size.restype = sz
            l.situ_moe_lora_backward_workspace_size.argtypes = [i32, i32, i32, i32]
            l.situ_moe_lora.restype = ctypes.c_int
            l.situ_moe_lora.argtypes = [ctypes.POINTER(SituLoraArgs), vp, sz, vp]
            l.situ_moe_lora_backward.restype = ctypes.c_int
            l.situ_moe_lora_backward.argtypes = [ctypes.POINTER(SituLoraBackwardArgs), vp, sz, vp]
            _lib = l
    return _lib


def status_string(status: int) -> str:
    return lib().situ_status_string(status).decode()


def _check(fn: str, status: int) -> None:
    if status != SITU_OK:
        raise SituError(fn, status)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def situ_moe_permute_workspace_size(T: int, top_k: int, num_local_experts: int) -> int:
    return lib().situ_moe_permute_workspace_size(T, top_k, num_local_experts)


def situ_moe_permute(topk_ids: torch.Tensor, num_experts_total: int, num_local_experts: int,
                     local_expert_offset: int, stream=None):
    """Returns (expert_counts, expert_offsets, permuted_src, slot_to_row)."""
    T, K = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty(num_local_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_local_experts + 1, dtype=torch.int32, device=dev)
    psrc = torch.empty(max(T * K, 1), dtype=torch.int32, device=dev)
    s2r = torch.empty(max(T * K, 1), dtype=torch.int32, device=dev)
    nbytes = situ_moe_permute_workspace_size(T, K, num_local_experts)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _check("situ_moe_permute", lib().situ_moe_permute(
        _p(topk_ids.contiguous()), T, K, num_experts_total, num_local_experts, local_expert_offset,
        _p(counts), _p(offsets), _p(psrc), _p(s2r), _p(ws), ws.numel(), _stream(stream)))
    return counts, offsets, psrc[:T * K], s2r[:T * K]


def situ_moe_permute_noalloc(topk_ids: torch.Tensor, num_experts_total: int,
                             num_local_experts: int, local_expert_offset: int, out=None,
                             stream=None):
    """situ_moe_permute with the library's fixed scratch instead of a
    workspace.  ``out`` = (counts, offsets, permuted_src, slot_to_row)
    preallocated by the caller; without it they are allocated here with torch
    (the C entry point itself never allocates)."""
    T, K = topk_ids.shape
    dev = topk_ids.device
    if topk_ids.dtype != torch.int32:
        raise TypeError("topk_ids must be int32")
    topk_ids = topk_ids.contiguous()   # a strided view would be read as if packed
    if out is None:
        out = (torch.empty(num_local_experts, dtype=torch.int32, device=dev),
               torch.empty(num_local_experts + 1, dtype=torch.int32, device=dev),
               torch.empty(max(T * K, 1), dtype=torch.int32, device=dev),
               torch.empty(max(T * K, 1), dtype=torch.int32, device=dev))
    counts, offsets, psrc, s2r = out
    # the kernels write every element of these: check what they will be given
    for t, n, what in ((counts, num_local_experts, "expert_counts"),
                       (offsets, num_local_experts + 1, "expert_offsets"),
                       (psrc, T * K, "permuted_src"), (s2r, T * K, "slot_to_row")):
        if t.dtype != torch.int32 or t.device != dev or not t.is_contiguous() or t.numel() < n:
            raise ValueError(f"{what}: needs a contiguous int32 tensor of >= {n} elements on {dev}")
    _check("situ_moe_permute_noalloc", lib().situ_moe_permute_noalloc(
        _p(topk_ids), T, K, num_experts_total, num_local_experts, local_expert_offset,
        _p(counts), _p(offsets), _p(psrc), _p(s2r), _stream(stream)))
    return counts, offsets, psrc[:T * K], s2r[:T * K]


def situ_moe_route_topk(router_logits: torch.Tensor, top_k: int, renormalize: bool = True, stream=None,
                        out=None):
    """Router logits fp32 [T, E] -> (int32 topk_ids [T, K], fp32 topk_weights
    [T, K]): the K largest logits (ties to the lower ID) and a softmax over
    them (renormalize) or their softmax probabilities over all E."""
    if router_logits.dtype != torch.float32:
        raise TypeError("router_logits must be fp32")
    logits = router_logits.contiguous()
    T, E = logits.shape
    if out is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    else:
        ids, w = out
    _check("situ_moe_route_topk", lib().situ_moe_route_topk(
        _p(logits), T, E, int(top_k), 1 if renormalize else 0, _p(ids), _p(w), _stream(stream)))
    return ids, w


def situ_moe_quant_mxfp8(x_bf16: torch.Tensor, stream=None, out=None):
    """bf16 [T,H] -> (E4M3 uint8 [T,H], UE8M0 uint8 [T,H/32])."""
    T, H = x_bf16.shape
    if out is None:
        q = torch.empty((T, H), dtype=torch.uint8, device=x_bf16.device)
        s = torch.empty((T, H // 32), dtype=torch.uint8, device=x_bf16.device)
    else:
        q, s = out
    _check("situ_moe_quant_mxfp8", lib().situ_moe_quant_mxfp8(
        _p(x_bf16), T, H, _p(q), _p(s), _stream(stream)))
    return q, s


def situ_moe_quant_nvfp4(x_bf16: torch.Tensor, stream=None, out=None):
    """bf16 [T,H] -> (packed E2M1 uint8 [T,H/2], E4M3 uint8 [T,H/16], fp32 [T])."""
    T, H = x_bf16.shape
    if out is None:
        q = torch.empty((T, H // 2), dtype=torch.uint8, device=x_bf16.device)
        s = torch.empty((T, H // 16), dtype=torch.uint8, device=x_bf16.device)
        g = torch.empty((T,), dtype=torch.float32, device=x_bf16.device)
    else:
        q, s, g = out
    _check("situ_moe_quant_nvfp4", lib().situ_moe_quant_nvfp4(
        _p(x_bf16), T, H, _p(q), _p(s), _p(g), _stream(stream)))
    return q, s, g


def make_args(*, T, H, I, num_experts_total, num_local_experts, local_expert_offset, top_k,
              act_dtype, weight_dtype, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale,
              gemm1_alpha, gemm1_beta, out, hidden_states=None, hidden_states_q=None,
              hidden_states_scale=None, hidden_states_gscale=None, w1_gscale=None, w2_gscale=None,
              g1_alphas=None, g1_alphas_up=None, g2_alphas=None) -> SituMoeArgs:
    a = SituMoeArgs(T=T, H=H, I=I, num_experts_total=num_experts_total,
                    num_local_experts=num_local_experts, local_expert_offset=local_expert_offset,
                    top_k=top_k, act_dtype=act_dtype, weight_dtype=weight_dtype)
    a.tactic[0] = a.tactic[1] = -1   # auto
    for name, t in dict(hidden_states=hidden_states, hidden_states_q=hidden_states_q,
                        hidden_states_scale=hidden_states_scale,
                        hidden_states_gscale=hidden_states_gscale, topk_ids=topk_ids,
                        topk_weights=topk_weights, w1=w1, w1_scale=w1_scale, w1_gscale=w1_gscale,
                        w2=w2, w2_scale=w2_scale, w2_gscale=w2_gscale, gemm1_alpha=gemm1_alpha,
                        gemm1_beta=gemm1_beta, g1_alphas=g1_alphas, g1_alphas_up=g1_alphas_up,
                        g2_alphas=g2_alphas, out=out).items():
        setattr(a, name, None if t is None else t.data_ptr())
    return a


def situ_moe_workspace_size(args: SituMoeArgs) -> int:
    return lib().situ_moe_workspace_size(ctypes.byref(args))


def situ_moe_packed_scales_size(args: SituMoeArgs) -> int:
    return lib().situ_moe_packed_scales_size(ctypes.byref(args))


def situ_moe_pack_scales(args: SituMoeArgs, packed: torch.Tensor, stream=None) -> None:
    """Packs the weight scales of ``args`` into ``packed`` (uint8 device
    tensor of at least situ_moe_packed_scales_size bytes)."""
    _check("situ_moe_pack_scales", lib().situ_moe_pack_scales(
        ctypes.byref(args), _p(packed), packed.numel() * packed.element_size(), _stream(stream)))


def situ_moe_forward_launches(args: SituMoeArgs) -> int:
    """Kernels situ_moe_forward enqueues for ``args`` (-1: invalid)."""
    return lib().situ_moe_forward_launches(ctypes.byref(args))


def situ_moe_forward(args: SituMoeArgs, workspace: torch.Tensor, stream=None) -> None:
    _check("situ_moe_forward", lib().situ_moe_forward(
        ctypes.byref(args), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


SITU_SELFTEST_WAIT_CODE = 99   # include/situ_moe.h


def situ_moe_wait_selftest(status: torch.Tensor, stream=None) -> None:
    """One bounded device wait made to run out (the failure path): after the
    wait limit the kernel records SITU_SELFTEST_WAIT_CODE in ``status`` (an
    int32 tensor on the device, zeroed by the caller) and returns."""
    _check("situ_moe_wait_selftest", lib().situ_moe_wait_selftest(_p(status), _stream(stream)))


def situ_moe_forward_wait_test(args: SituMoeArgs, workspace: torch.Tensor, skip_stage: int, wait_us: int,
                               stream=None) -> None:
    """situ_moe_forward whose FC1 (block-scaled decode tiles) leaves K stage
    ``skip_stage`` of CTA 0 unissued, with every wait limited to ``wait_us``:
    the failure path on purpose (read the outcome with situ_moe_device_status)."""
    _check("situ_moe_forward_wait_test", lib().situ_moe_forward_wait_test(
        ctypes.byref(args), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream),
        int(skip_stage), int(wait_us)))


SITU_TC_MXF8F6F4, SITU_TC_MXF4NVF4, SITU_TC_BF16 = 0, 1, 2
TC_KIND_NAMES = {SITU_TC_MXF8F6F4: "mxf8f6f4", SITU_TC_MXF4NVF4: "mxf4nvf4", SITU_TC_BF16: "bf16"}


def situ_tc_peak(kind: int, mmas_per_sm: int, status: torch.Tensor, stream=None) -> float:
    """Enqueues the MMA-throughput kernel of ``kind`` (SITU_TC_*) with
    ``mmas_per_sm`` MMAs per SM; returns the launch's dense FLOPs.  ``status``
    is an int32 device tensor zeroed by the caller (98 after a timed-out wait)."""
    flops = ctypes.c_double(0.0)
    _check("situ_tc_peak", lib().situ_tc_peak(int(kind), int(mmas_per_sm), _p(status),
                                              ctypes.byref(flops), _stream(stream)))
    return float(flops.value)


def situ_moe_device_status(args: SituMoeArgs, workspace: torch.Tensor, stream=None) -> int:
    """Waits for ``stream`` and returns the device status word of the last
    forward run with this workspace: 0, or the code of the first bounded
    wait a kernel gave up (the C call's SITU_ERR_DEVICE_TIMEOUT is not
    raised, it is reported through the code)."""
    code = ctypes.c_int32(0)
    st = lib().situ_moe_device_status(ctypes.byref(args), _p(workspace), _stream(stream),
                                      ctypes.byref(code))
    if st not in (0, SITU_ERR_DEVICE_TIMEOUT):
        _check("situ_moe_device_status", st)
    return int(code.value)


PROFILE_STAGES = ("permute", "gather", "fc1", "fc2", "combine")


def situ_moe_forward_profiled(args: SituMoeArgs, workspace: torch.Tensor, events, stream=None):
    """situ_moe_forward recording ``events`` (len(PROFILE_STAGES) + 1
    torch.cuda.Event objects with timing enabled) around each stage."""
    assert len(events) == len(PROFILE_STAGES) + 1
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check("situ_moe_forward_profiled", lib().situ_moe_forward_profiled(
        ctypes.byref(args), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream), arr))


# ---------------------------------------------------------------------------
# expert products with 16-bit and with E4M3 weights
#
# Each call enqueues on ``stream`` (default: the current stream of the
# operands' device); results and copies are allocated on that stream.  The
# caller orders it after the work that makes the operands, and before the work
# that reads the results; the operands may be dropped at once.  A
# first call on a device waits for it once (its status word), so it does not
# belong inside a graph capture.
# ---------------------------------------------------------------------------

_DTYPES = {torch.bfloat16: SITU_DT_BF16, torch.float16: SITU_DT_F16, torch.float32: SITU_DT_F32}
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_gemm_status = {}


def _status_word(index: int) -> torch.Tensor:
    """The status word that this process's products on GPU ``index`` share."""
    t = _gemm_status.get(index)
    if t is None:
        with torch.cuda.device(index):
            t = torch.zeros(1, dtype=torch.int32, device=f"cuda:{index}")
            torch.cuda.synchronize()   # once per device: zero before any stream uses it
        t = _gemm_status.setdefault(index, t)
    return t


def situ_moe_gemm_status(device=None, reset: bool = False) -> int:
    """0, or the code of the first bounded wait that a product
    (situ_moe_grouped_gemm*, situ_moe_fp8*_gemm, situ_moe_lora*) on ``device``
    gave up; until it is reset the products there do no work.  Waits for the
    device."""
    device = torch.device("cuda" if device is None else device)
    index = torch.cuda.current_device() if device.index is None else device.index
    torch.cuda.synchronize(index)
    t = _status_word(index)
    code = int(t.item())
    if reset and code:
        t.zero_()
        torch.cuda.synchronize(index)
    return code


# The short calls (a decode step's) take the GPU less time than their
# marshalling takes the host, so what every call passes through is kept short:
# where this torch has them, the direct forms of torch.cuda.current_stream (0.1
# for 2.9 us here) and of torch.empty (0.9 for 2.3 us), and no helper calls for
# operands that need none.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _empty(shape, strides, dtype, index: int) -> torch.Tensor:
    """An uninitialised packed tensor on GPU ``index``."""
    if _empty_cuda is not None and _current_device() == index:
        return _empty_cuda(shape, strides, dtype)
    return torch.empty(shape, dtype=dtype, device=f"cuda:{index}")


def _enqueue(name: str, index: int, *args) -> None:
    """Calls the C entry point ``name`` on GPU ``index`` and its current stream."""
    fn = getattr(_lib or lib(), name)
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(name, status)


def _on_stream(stream, f, x: torch.Tensor, *args, **kw):
    """f(x, *args, **kw) with ``stream`` current: what it allocates and copies
    belongs to that stream too, and the memory of operands that belong to
    another is not given to anyone else before this work is done."""
    if stream.device != x.device:
        raise ValueError(f"a stream of {stream.device} for operands on {x.device}")
    with torch.cuda.stream(stream):
        result = f(x, *args, **kw)
    for t in (x, *args, *kw.values()):
        for u in t if isinstance(t, (tuple, list)) else (t,):
            if isinstance(u, torch.Tensor) and u.is_cuda:
                u.record_stream(stream)
    return result


def _rows(t: torch.Tensor, unit: int):
    """(tensor, pointer, elements between rows) of ``t`` [R, C]: itself where
    the kernels can read it in place (columns packed, rows a multiple of
    ``unit`` elements apart, 16-byte aligned), else a copy."""
    R, C = t.shape
    p = t.data_ptr()
    if not p & 15:
        if t.is_contiguous():
            return t, p, C
        s0, s1 = t.stride()
        if s1 == 1 and s0 >= C and s0 % unit == 0:
            return t, p, s0
    t = t.clone(memory_format=torch.contiguous_format)
    return t, t.data_ptr(), C


def _packed(t: torch.Tensor):
    """(tensor, pointer) of ``t`` contiguous and 16-byte aligned: itself or a copy."""
    p = t.data_ptr()
    if not t.is_contiguous() or p & 15:
        t = t.clone(memory_format=torch.contiguous_format)
        p = t.data_ptr()
    return t, p


def _weights(t: torch.Tensor, unit: int):
    """(tensor, pointer, elements between rows, between experts; 0 and 0:
    contiguous) of weights [E, N, K] or [N, K]: itself where the kernels can
    read it in place (a part of a larger array, as one half of gate and up
    weights held together), else a copy."""
    p = t.data_ptr()
    if not p & 15:
        if t.is_contiguous():
            return t, p, 0, 0
        N, K = t.shape[-2:]
        ld = t.stride(-2)
        if t.stride(-1) == 1 and ld >= K and ld % unit == 0:
            se = N * ld if t.dim() == 2 or t.shape[0] == 1 else t.stride(0)
            if se >= N * ld and se % ld == 0:
                return t, p, ld, se
    t = t.clone(memory_format=torch.contiguous_format)
    return t, t.data_ptr(), 0, 0


def _given(out: torch.Tensor, shape, dtype, index: int, unit: int) -> int:
    """The elements between the rows of a caller's ``out``, after its checks."""
    if tuple(out.shape) != shape or out.dtype is not dtype or out.get_device() != index:
        raise ValueError(f"out: needs {dtype} {shape} on cuda:{index}")
    if not out.data_ptr() & 15:
        if out.is_contiguous():
            return shape[-1]
        if len(shape) == 2 and out.stride(1) == 1 and out.stride(0) >= shape[1] and out.stride(0) % unit == 0:
            return out.stride(0)
    raise ValueError("out: needs 16-byte aligned rows, packed along the last dimension")


def _groups(offsets: torch.Tensor, index: int) -> int:
    """The number of groups that ``offsets`` bounds."""
    if offsets.dtype is not torch.int32 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise TypeError("offsets must be int32 [E + 1]")
    if offsets.get_device() != index:
        raise ValueError(f"offsets on {offsets.device}, the operands on cuda:{index}")
    return offsets.shape[0] - 1


def _too_large(*sizes):
    return ValueError(f"sizes {sizes} must be below 2^31")


def _grouped(a, direction, b, offsets, S, E, N, K, out, shape, strides, out_dtype, accumulate, zero_rest):
    index, dtype = a.get_device(), a.dtype
    if (S | E | N | K) >> 31:   # ctypes would cut them to 32 bits
        raise _too_large(S, E, N, K)
    if index < 0 or b.get_device() != index:
        raise ValueError(f"the operands must be on one CUDA device, not on {a.device} and {b.device}")
    if dtype is not torch.bfloat16 and dtype is not torch.float16 or b.dtype is not dtype:
        raise TypeError("the operands must be both bf16 or both f16")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else dtype
    if out_dtype is not dtype and out_dtype is not torch.float32:
        raise TypeError("the output must be of the operands' type or fp32")
    if _groups(offsets, index) != E:
        raise ValueError("weights must be [E, N, K] with offsets [E + 1]")
    if out is None:
        out, ldo = _empty(shape, strides, out_dtype, index), shape[-1]
    else:
        ldo = _given(out, shape, out_dtype, index, 8)
    if not offsets.is_contiguous():
        offsets = offsets.contiguous()
    a, pa, lda = _rows(a, 8)
    ldb = ldw = stride_w = 0
    if direction == SITU_GROUPED_WGRAD:
        b, pb, ldb = _rows(b, 8)
    else:
        b, pb, ldw, stride_w = _weights(b, 8)
    args = SituGroupedGemmArgs(direction, _DTYPES[dtype], _DTYPES[out_dtype], S, N, K, E, accumulate, not zero_rest,
                               pa, lda, pb, ldb, offsets.data_ptr(), out.data_ptr(), ldo, _status_word(index).data_ptr(),
                               ldw, stride_w)
    _enqueue("situ_moe_grouped_gemm", index, ctypes.byref(args))
    return out


def situ_moe_grouped_gemm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, out=None, out_dtype=None,
                          zero_rest: bool = True, stream=None) -> torch.Tensor:
    """y[r] = x[r] @ w[e].T for the rows r of each expert e: x [S, K] sorted by
    expert, w [E, N, K] of the same 16-bit type (or one expert's [N, K]),
    offsets int32 [E + 1] (as situ_moe_permute returns them).  Rows of no expert
    give zeros, or are left unwritten with ``zero_rest=False``.  Rows, of
    weights too, may be strided; a layout that the kernels cannot read in place
    (columns apart, rows off 16 bytes, experts broadcast) is copied first, in
    each of these calls."""
    if stream is not None:
        return _on_stream(stream, situ_moe_grouped_gemm, x, w, offsets, out=out, out_dtype=out_dtype, zero_rest=zero_rest)
    E, N, K = w.shape if w.dim() == 3 else (1, *w.shape)
    S, Kx = x.shape
    if Kx != K:
        raise ValueError("x must be [S, K]")
    return _grouped(x, SITU_GROUPED_FORWARD, w, offsets, S, E, N, K, out, (S, N), (N, 1), out_dtype, False, zero_rest)


def situ_moe_grouped_gemm_dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, out=None,
                                out_dtype=None, zero_rest: bool = True, stream=None) -> torch.Tensor:
    """The gradient of situ_moe_grouped_gemm's x: dx[r] = dy[r] @ w[e], [S, K]."""
    if stream is not None:
        return _on_stream(stream, situ_moe_grouped_gemm_dgrad, dy, w, offsets, out=out, out_dtype=out_dtype,
                          zero_rest=zero_rest)
    E, N, K = w.shape if w.dim() == 3 else (1, *w.shape)
    S, Ny = dy.shape
    if Ny != N:
        raise ValueError("dy must be [S, N]")
    return _grouped(dy, SITU_GROUPED_DGRAD, w, offsets, S, E, N, K, out, (S, K), (K, 1), out_dtype, False, zero_rest)


def situ_moe_grouped_gemm_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, *, out=None,
                                out_dtype=None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """The gradient of its w: dw[e] = dy[rows of e].T @ x[rows of e], [E, N, K];
    zeros for an expert without rows.  ``accumulate`` adds to ``out``."""
    if stream is not None:
        return _on_stream(stream, situ_moe_grouped_gemm_wgrad, dy, x, offsets, out=out, out_dtype=out_dtype,
                          accumulate=accumulate)
    S, N = dy.shape
    Sx, K = x.shape
    if S != Sx:
        raise ValueError("dy must be [S, N] and x [S, K]")
    if accumulate and out is None:
        raise ValueError("accumulate adds to out: none given")
    E = offsets.numel() - 1
    return _grouped(dy, SITU_GROUPED_WGRAD, x, offsets, S, E, N, K, out, (E, N, K), (N * K, K, 1), out_dtype, accumulate,
                    True)


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return situ_moe_grouped_gemm(x, w, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dx = situ_moe_grouped_gemm_dgrad(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = situ_moe_grouped_gemm_wgrad(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
    """situ_moe_grouped_gemm for training: differentiable in x [S, K] and
    w [E, N, K]."""
    if w.dim() != 3:
        raise ValueError("w must be [E, N, K]")
    return _GroupedLinear.apply(x, w, offsets)


def situ_moe_quant_fp8(x: torch.Tensor, block_rows: int = 1, *, out=None, stream=None):
    """bf16, f16 or fp32 [R, K] or [E, R, K] -> (E4M3 uint8 of x's shape, fp32
    scales per block of 128): block_rows 1, a scale per row and 128 columns
    (activations); 128, one per 128 x 128 block (weights)."""
    if stream is not None:
        return _on_stream(stream, situ_moe_quant_fp8, x, block_rows, out=out)
    index, dtype, dim = x.get_device(), _DTYPES.get(x.dtype), x.dim()
    if dtype is None:
        raise TypeError("x must be bf16, f16 or fp32")
    if max(x.shape) >> 31:
        raise _too_large(*x.shape)
    if index < 0:
        raise ValueError("x must be a CUDA tensor")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    if dim == 2:
        E, (R, K) = 1, x.shape
        nr, nk = -(-R // block_rows), -(-K // 128)
        x, px, ldx = _rows(x, 4 if dtype == SITU_DT_F32 else 8)
        shape, strides, dims, dstrides = (R, K), (K, 1), (nr, nk), (nk, 1)
    elif dim == 3:
        E, R, K = x.shape
        nr, nk = -(-R // block_rows), -(-K // 128)
        x, px = _packed(x)
        ldx = K
        shape, strides, dims, dstrides = (E, R, K), (R * K, K, 1), (E, nr, nk), (nr * nk, nk, 1)
    else:
        raise ValueError("x must be [R, K] or [E, R, K]")
    if out is None:
        q, scale = _empty(shape, strides, torch.uint8, index), _empty(dims, dstrides, torch.float32, index)
    else:
        q, scale = out
        for t, want, dts, what in ((q, shape, _E4M3, "q"), (scale, dims, (torch.float32,), "scale")):
            if tuple(t.shape) != want or t.dtype not in dts or t.get_device() != index or not t.is_contiguous():
                raise ValueError(f"{what}: needs a contiguous {dts[0]} tensor {want} on cuda:{index}")
    _enqueue("situ_moe_quant_fp8", index, px, dtype, E, R, K, ldx, block_rows, q.data_ptr(), scale.data_ptr())
    return q, scale


def _fp8_gemm(x_q, x_scale, w_q, w_scale, E, N, K, offsets, out, out_dtype, zero_rest):
    index = x_q.get_device()
    S, Kx = x_q.shape
    if (S | E | N | K) >> 31:
        raise _too_large(S, E, N, K)
    if index < 0 or x_scale.get_device() != index or w_q.get_device() != index or w_scale.get_device() != index:
        raise ValueError("the operands must be on one CUDA device")
    if x_q.dtype not in _E4M3 or w_q.dtype not in _E4M3:
        raise TypeError("x_q and w_q must hold E4M3 codes (uint8 or float8_e4m3fn)")
    if x_scale.dtype is not torch.float32 or w_scale.dtype is not torch.float32:
        raise TypeError("the scales must be fp32")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise TypeError("the output must be bf16 or fp32")
    nkb, nrb = -(-K // 128), -(-N // 128)
    if Kx != K or x_scale.shape != (S, nkb):
        raise ValueError(f"needs x_q [S, {K}] and x_scale [S, {nkb}]")
    if w_scale.shape != (E, nrb, nkb) and (E != 1 or w_scale.shape != (nrb, nkb)):
        raise ValueError(f"needs w_scale {(E, nrb, nkb)}")
    if offsets is None:
        poff = None
    else:
        if _groups(offsets, index) != E:
            raise ValueError("weights must be [E, N, K] with offsets [E + 1]")
        if not offsets.is_contiguous():
            offsets = offsets.contiguous()
        poff = offsets.data_ptr()
    if out is None:
        out, ldo = _empty((S, N), (N, 1), out_dtype, index), N
    else:
        ldo = _given(out, (S, N), out_dtype, index, 8)
    x_q, px, ldx = _rows(x_q, 16)
    w_q, pw, ldw, stride_w = _weights(w_q, 16)
    if not x_scale.is_contiguous():
        x_scale = x_scale.contiguous()
    if not w_scale.is_contiguous():
        w_scale = w_scale.contiguous()
    args = SituFp8GemmArgs(_DTYPES[out_dtype], S, N, K, E, not zero_rest, px, ldx, x_scale.data_ptr(), pw,
                           w_scale.data_ptr(), poff, out.data_ptr(), ldo, _status_word(index).data_ptr(), ldw, stride_w)
    _enqueue("situ_moe_fp8_gemm", index, ctypes.byref(args))
    return out


def situ_moe_fp8_gemm(x_q: torch.Tensor, x_scale: torch.Tensor, w_q: torch.Tensor, w_scale: torch.Tensor, *,
                      out=None, out_dtype=None, stream=None) -> torch.Tensor:
    """x @ w.T of operands quantised by situ_moe_quant_fp8: x_q [S, K] with a
    scale per row and 128 columns, w_q [N, K] with one per 128 x 128 block;
    bf16 (default) or fp32 [S, N]."""
    if stream is not None:
        return _on_stream(stream, situ_moe_fp8_gemm, x_q, x_scale, w_q, w_scale, out=out, out_dtype=out_dtype)
    if w_scale.dim() != 2:
        raise ValueError("w_q must be [N, K] and w_scale [ceil(N/128), ceil(K/128)]")
    N, K = w_q.shape
    return _fp8_gemm(x_q, x_scale, w_q, w_scale, 1, N, K, None, out, out_dtype, True)


def situ_moe_fp8_grouped_gemm(x_q: torch.Tensor, x_scale: torch.Tensor, w_q: torch.Tensor, w_scale: torch.Tensor,
                              offsets: torch.Tensor, *, out=None, out_dtype=None, zero_rest: bool = True,
                              stream=None) -> torch.Tensor:
    """The same per expert: rows of x_q sorted by expert, w_q [E, N, K] (or one
    expert's [N, K]), offsets int32 [E + 1].  Rows of no expert give zeros, or
    are left unwritten with ``zero_rest=False``."""
    if stream is not None:
        return _on_stream(stream, situ_moe_fp8_grouped_gemm, x_q, x_scale, w_q, w_scale, offsets, out=out,
                          out_dtype=out_dtype, zero_rest=zero_rest)
    E, N, K = w_q.shape if w_q.dim() == 3 else (1, *w_q.shape)
    return _fp8_gemm(x_q, x_scale, w_q, w_scale, E, N, K, offsets, out, out_dtype, zero_rest)


# ---------------------------------------------------------------------------
# fine-tuning: the router's balance loss, the gated activation with its input
# kept in 8 bits, low-rank adapters
#
# Streams, devices and copies are as for the expert products above.  None of
# these calls waits for the device, except a first situ_moe_lora or
# situ_moe_lora_backward on it (the products' status word, which they share): that
# does not belong inside a graph capture.
# ---------------------------------------------------------------------------

# workspace sizes of shapes already seen: a call into the library less
@functools.lru_cache(maxsize=4096)
def _balance_bytes(T, E, index):
    return _size("situ_moe_balance_loss_workspace_size", index, T, E)


@functools.lru_cache(maxsize=4096)
def _lora_bytes(S, K, N, r, n, index):
    return _size("situ_moe_lora_workspace_size", index, S, K, N, r, n)


@functools.lru_cache(maxsize=4096)
def _lora_backward_bytes(S, K, N, r, index):
    return _size("situ_moe_lora_backward_workspace_size", index, S, K, N, r)


def _size(name, index, *args) -> int:
    with torch.cuda.device(index):
        return getattr(_lib or lib(), name)(*args)


def _new(index: int):
    """_empty on GPU ``index``, the device looked at once for several tensors."""
    if _empty_cuda is not None and _current_device() == index:
        return _empty_cuda
    return lambda shape, strides, dtype: torch.empty(shape, dtype=dtype, device=f"cuda:{index}")


def _scratch(n: int, new):
    """(tensor or None, pointer or None) of n bytes; the caller keeps the tensor until the call is enqueued."""
    if n == 0:
        return None, None
    t = new((n,), (1,), torch.uint8)
    return t, t.data_ptr()


def _on_device(index: int, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name} on {t.device}, the operands on cuda:{index}")


def _vector(t: torch.Tensor, dtype, n: int, name: str, index: int) -> torch.Tensor:
    """``t`` as a contiguous [n] of ``dtype``, checked."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != (n,):
        raise ValueError(f"{name} must be [{n}], not {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} on {t.device}, the operands on cuda:{index}")
    return t if t.is_contiguous() else t.contiguous()


def _logits(t: torch.Tensor):
    """(tensor, elements between rows) of router logits: itself or a copy."""
    if t.is_contiguous():
        return t, t.shape[1]
    if t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t, t.stride(0)
    return t.contiguous(), t.shape[1]


def _router(router_logits, topk_ids, mask):
    """Checks what both router calls take: (logits, ld, ids, mask, index, T, E, k)."""
    index = router_logits.get_device()
    if router_logits.dtype is not torch.float32:
        raise TypeError("router_logits must be fp32")
    if topk_ids.dtype is not torch.int32:
        raise TypeError("topk_ids must be int32")
    if router_logits.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != router_logits.shape[0]:
        raise ValueError("needs router_logits [T, E] and topk_ids [T, k]")
    if index < 0 or topk_ids.get_device() != index:
        raise ValueError(f"the operands must be on one CUDA device, not on {router_logits.device} and {topk_ids.device}")
    T, E = router_logits.shape
    k = topk_ids.shape[1]
    if (T | E | k) >> 31:
        raise _too_large(T, E, k)
    if mask is not None:
        mask = _vector(mask, torch.uint8 if mask.dtype is torch.uint8 else torch.bool, T, "mask", index)
    logits, ld = _logits(router_logits)
    return logits, ld, topk_ids if topk_ids.is_contiguous() else topk_ids.contiguous(), mask, index, T, E, k


def situ_moe_balance_loss(router_logits: torch.Tensor, topk_ids: torch.Tensor, *, mask=None, coef: float = 1.0,
                          stream=None):
    """The router's balance loss over the tokens that ``mask`` (bool or uint8
    [T]; None: all) leaves: coef * E * sum_e f_e P_e, f_e the share of the
    chosen slots that name expert e, P_e its mean softmax probability.  Returns
    (loss fp32 [], counts int32 [E] of the slots per expert, tokens int32 [1],
    row_stats fp32 [T, 2]), the last two for situ_moe_router_backward."""
    if stream is not None:
        return _on_stream(stream, situ_moe_balance_loss, router_logits, topk_ids, mask=mask, coef=coef)
    logits, ld, ids, mask, index, T, E, k = _router(router_logits, topk_ids, mask)
    new = _new(index)
    loss, counts = new((), (), torch.float32), new((E,), (1,), torch.int32)
    tokens, stats = new((1,), (1,), torch.int32), new((T, 2), (2, 1), torch.float32)
    n = _balance_bytes(T, E, index)
    ws, pws = _scratch(n, new)
    args = SituBalanceArgs(logits.data_ptr(), ld, ids.data_ptr(), None if mask is None else mask.data_ptr(), T, E, k, coef,
                           loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(), stats.data_ptr())
    _enqueue("situ_moe_balance_loss", index, ctypes.byref(args), pws, n)
    return loss, counts, tokens, stats


def situ_moe_router_backward(router_logits: torch.Tensor, topk_ids: torch.Tensor, counts, tokens, row_stats, *,
                             dloss=None, coef: float = 1.0, mask=None, topk_weights=None, dweights=None,
                             renormalize: bool = True, out=None, stream=None) -> torch.Tensor:
    """The gradient fp32 [T, E] of the router's logits, from that of the balance
    loss (``dloss``, one fp32 on the device) with the forward's coef and mask,
    and those of situ_moe_route_topk's weights (``dweights`` [T, k] beside
    ``topk_weights``, with its ``renormalize``); either may be None."""
    if stream is not None:
        return _on_stream(stream, situ_moe_router_backward, router_logits, topk_ids, counts, tokens, row_stats,
                          dloss=dloss, coef=coef, mask=mask, topk_weights=topk_weights, dweights=dweights,
                          renormalize=renormalize, out=out)
    logits, ld, ids, mask, index, T, E, k = _router(router_logits, topk_ids, mask)
    if (row_stats.shape != (T, 2) or row_stats.dtype is not torch.float32 or not row_stats.is_contiguous()
            or row_stats.get_device() != index):
        raise ValueError(f"row_stats must be contiguous fp32 [{T}, 2] on cuda:{index}")
    pl = pc = pt = pw = pd = None
    if dloss is not None:
        counts, tokens = _vector(counts, torch.int32, E, "counts", index), _vector(tokens, torch.int32, 1, "tokens", index)
        if dloss.dtype is not torch.float32 or dloss.numel() != 1 or dloss.get_device() != index:
            raise ValueError(f"dloss must be one fp32 on cuda:{index}")
        pl, pc, pt = dloss.data_ptr(), counts.data_ptr(), tokens.data_ptr()
    if dweights is not None:
        if topk_weights is None:
            raise ValueError("dweights needs the topk_weights")
        for name, t in (("topk_weights", topk_weights), ("dweights", dweights)):
            if t.dtype is not torch.float32 or t.shape != (T, k) or t.get_device() != index:
                raise ValueError(f"{name} must be fp32 [{T}, {k}] on cuda:{index}")
        if not topk_weights.is_contiguous():
            topk_weights = topk_weights.contiguous()
        if not dweights.is_contiguous():
            dweights = dweights.contiguous()
        pw, pd = topk_weights.data_ptr(), dweights.data_ptr()
    if out is None:
        out, ldo = _empty((T, E), (E, 1), torch.float32, index), E
    else:
        ldo = _given(out, (T, E), torch.float32, index, 1)
    args = SituRouterBackwardArgs(logits.data_ptr(), ld, ids.data_ptr(), None if mask is None else mask.data_ptr(), T, E, k,
                                  1 if renormalize else 0, coef, pc, pt, row_stats.data_ptr(), pl, pw, pd, out.data_ptr(),
                                  ldo)
    _enqueue("situ_moe_router_backward", index, ctypes.byref(args))
    return out


def _constant(**tensors) -> None:
    """Refuses what a gradient is asked for and none is made of."""
    for name, t in tensors.items():
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} gets no gradient here: detach it, or clear its requires_grad")


def _graphed(f, *args):
    """f(*args) of an autograd function.  torch adds a leaf's gradient on the
    stream on which the first of its living graphs was built.  A backward pass
    captured elsewhere draws that stream into the capture, which is fine but for
    the legacy default stream: that can end the process, so the captured forward
    pass is refused."""
    nodes = []
    if torch.is_grad_enabled():
        for t in args:
            if isinstance(t, torch.Tensor) and t.is_cuda and t.requires_grad and t.is_leaf:
                node, stream = torch.autograd.graph.get_gradient_edge(t).node, _raw_stream(t.get_device())
                nodes.append(node)   # alive until f's graph holds it
                if node.metadata.setdefault("situ_moe stream", stream) == 0 != stream and torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("captured while a graph of the same leaf, built on the default stream, is alive: drop what "
                                       "holds it (outputs, losses), or build it under a side stream, as a wrapper that keeps "
                                       "its leaves' nodes has to be")
    return f(*args)


class _BalancedRoute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, router_logits, top_k, renormalize, mask, coef):
        with torch.cuda.device(router_logits.device):
            ids, weights = situ_moe_route_topk(router_logits, top_k, renormalize)
            loss, counts, tokens, stats = situ_moe_balance_loss(router_logits, ids, mask=mask, coef=coef)
        ctx.save_for_backward(router_logits, ids, weights, counts, tokens, stats, mask)
        ctx.renormalize, ctx.coef = renormalize, coef
        ctx.mark_non_differentiable(ids, counts)
        ctx.set_materialize_grads(False)
        return ids, weights, counts, loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _ids, dweights, _counts, dloss):
        logits, ids, weights, counts, tokens, stats, mask = ctx.saved_tensors
        if dweights is None and dloss is None:
            return None, None, None, None, None
        d = situ_moe_router_backward(logits, ids, counts, tokens, stats, dloss=dloss, coef=ctx.coef, mask=mask,
                                     topk_weights=weights, dweights=dweights, renormalize=ctx.renormalize)
        return d, None, None, None, None


def balanced_route(router_logits: torch.Tensor, top_k: int, *, renormalize: bool = True, mask=None, coef: float = 0.01):
    """situ_moe_route_topk for training: (topk_ids, topk_weights, counts, loss),
    the weights and the balance loss differentiable in the logits."""
    return _graphed(_BalancedRoute.apply, router_logits, top_k, renormalize, mask, coef)


def situ_moe_save_mxfp8(x: torch.Tensor, *, out=None, stream=None):
    """16-bit activations [S, K] kept in 8 bits: (E4M3 uint8 [S, K], UE8M0 uint8
    [S, ceil(K/32)])."""
    if stream is not None:
        return _on_stream(stream, situ_moe_save_mxfp8, x, out=out)
    index = x.get_device()
    if x.dtype is not torch.bfloat16 and x.dtype is not torch.float16:
        raise TypeError("x must be bf16 or f16")
    if x.dim() != 2 or index < 0:
        raise ValueError("x must be [S, K] on a CUDA device")
    S, K = x.shape
    if (S | K) >> 31:
        raise _too_large(S, K)
    nk = -(-K // 32)
    x, px, ldx = _rows(x, 8)
    if out is None:
        new = _new(index)
        q, scale = new((S, K), (K, 1), torch.uint8), new((S, nk), (nk, 1), torch.uint8)
    else:
        q, scale = out
        for t, want, what in ((q, (S, K), "q"), (scale, (S, nk), "scale")):
            if tuple(t.shape) != want or t.dtype is not torch.uint8 or t.get_device() != index or not t.is_contiguous():
                raise ValueError(f"{what}: needs a contiguous uint8 tensor {want} on cuda:{index}")
    _enqueue("situ_moe_save_mxfp8", index, px, _DTYPES[x.dtype], S, K, ldx, q.data_ptr(), scale.data_ptr())
    return q, scale


def _kept(q, scale, S, K, blocks, index):
    """(q, scale) of a kept form, checked and contiguous."""
    if q.dtype not in _E4M3 or scale.dtype is not torch.uint8:
        raise TypeError("q must hold E4M3 codes (uint8 or float8_e4m3fn) and scale bytes")
    if q.shape != (S, K) or scale.shape != (S, blocks):
        raise ValueError(f"needs q [{S}, {K}] and scale [{S}, {blocks}]")
    if q.get_device() != index or scale.get_device() != index:
        raise ValueError(f"q on {q.device} and scale on {scale.device}, the operands on cuda:{index}")
    if not q.is_contiguous() or q.data_ptr() & 7:
        q = q.clone(memory_format=torch.contiguous_format)
    return q, scale if scale.is_contiguous() else scale.contiguous()


def situ_moe_restore_mxfp8(q: torch.Tensor, scale: torch.Tensor, dtype=torch.bfloat16, *, out=None,
                           stream=None) -> torch.Tensor:
    """What situ_moe_save_mxfp8 kept, as bf16, f16 or fp32 [S, K]."""
    if stream is not None:
        return _on_stream(stream, situ_moe_restore_mxfp8, q, scale, dtype, out=out)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be bf16, f16 or fp32")
    index = q.get_device()
    if q.dim() != 2 or index < 0:
        raise ValueError("q must be [S, K] on a CUDA device")
    S, K = q.shape
    if (S | K) >> 31:
        raise _too_large(S, K)
    q, scale = _kept(q, scale, S, K, -(-K // 32), index)
    if out is None:
        out, ldx = _empty((S, K), (K, 1), dtype, index), K
    else:
        ldx = _given(out, (S, K), dtype, index, 4 if dtype is torch.float32 else 8)
    _enqueue("situ_moe_restore_mxfp8", index, q.data_ptr(), scale.data_ptr(), _DTYPES[dtype], S, K, out.data_ptr(), ldx)
    return out


def _caps(p0, p1, offsets, index):
    """(p0, p1, offsets, their pointer, E) of the gated activation, checked."""
    E = 1 if offsets is None else _groups(offsets, index)
    p0, p1 = _vector(p0, torch.float32, E, "p0", index), _vector(p1, torch.float32, E, "p1", index)
    if offsets is not None and not offsets.is_contiguous():
        offsets = offsets.contiguous()
    return p0, p1, offsets, None if offsets is None else offsets.data_ptr(), E


def situ_moe_gated(gate_up: torch.Tensor, p0: torch.Tensor, p1: torch.Tensor, offsets=None, *,
                   activation: int = SITU_ACT_FN_SITU, save: bool = False, out=None, stream=None):
    """The layer's gated activation h [S, I] of 16-bit gate_up [S, 2I] (gate
    first): SITU with the caps p0 and p1, or SWIGLU_BIAS with alpha p0 and beta
    p1, fp32 [E] per expert of the rows that ``offsets`` [E + 1] bounds (None:
    [1], one for all).  Rows of no expert give zeros.  With ``save``: (h, q,
    scale), gate_up kept in 8 bits for situ_moe_gated_backward."""
    if stream is not None:
        return _on_stream(stream, situ_moe_gated, gate_up, p0, p1, offsets, activation=activation, save=save, out=out)
    index, dtype = gate_up.get_device(), gate_up.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("gate_up must be bf16 or f16")
    if gate_up.dim() != 2 or gate_up.shape[1] % 2 or index < 0:
        raise ValueError("gate_up must be [S, 2I] on a CUDA device")
    S, I = gate_up.shape[0], gate_up.shape[1] // 2
    if (S | 2 * I) >> 31:
        raise _too_large(S, 2 * I)
    p0, p1, offsets, poff, E = _caps(p0, p1, offsets, index)
    new = _new(index)
    x, px, ldx = _rows(gate_up, 8)
    if out is None:
        h, ldh = new((S, I), (I, 1), dtype), I
    else:
        h, ldh = out, _given(out, (S, I), dtype, index, 8)
    q = scale = pq = ps = None
    if save:
        nb = 2 * -(-I // 32)
        q, scale = new((S, 2 * I), (2 * I, 1), torch.uint8), new((S, nb), (nb, 1), torch.uint8)
        pq, ps = q.data_ptr(), scale.data_ptr()
    args = SituGatedArgs(_DTYPES[dtype], activation, S, I, E, px, ldx, p0.data_ptr(), p1.data_ptr(), poff, h.data_ptr(),
                         ldh, pq, ps, None, 0, None, 0)
    _enqueue("situ_moe_gated", index, ctypes.byref(args))
    return (h, q, scale) if save else h


def situ_moe_gated_backward(dh: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, p0: torch.Tensor, p1: torch.Tensor,
                            offsets=None, *, activation: int = SITU_ACT_FN_SITU, want_h: bool = False, out=None,
                            stream=None):
    """From dh [S, I] and what situ_moe_gated kept: (dgate_up [S, 2I], h [S, I]
    once more, or None without ``want_h``), both at the restored gate and up."""
    if stream is not None:
        return _on_stream(stream, situ_moe_gated_backward, dh, q, scale, p0, p1, offsets, activation=activation,
                          want_h=want_h, out=out)
    index, dtype = dh.get_device(), dh.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("dh must be bf16 or f16")
    if dh.dim() != 2 or index < 0:
        raise ValueError("dh must be [S, I] on a CUDA device")
    S, I = dh.shape
    if (S | 2 * I) >> 31:
        raise _too_large(S, 2 * I)
    q, scale = _kept(q, scale, S, 2 * I, 2 * -(-I // 32), index)
    p0, p1, offsets, poff, E = _caps(p0, p1, offsets, index)
    new = _new(index)
    dh, pdh, ldh = _rows(dh, 8)
    if out is None:
        out, ldo = new((S, 2 * I), (2 * I, 1), dtype), 2 * I
    else:
        ldo = _given(out, (S, 2 * I), dtype, index, 8)
    h = new((S, I), (I, 1), dtype) if want_h else None
    args = SituGatedArgs(_DTYPES[dtype], activation, S, I, E, None, 0, p0.data_ptr(), p1.data_ptr(), poff,
                         None if h is None else h.data_ptr(), I, q.data_ptr(), scale.data_ptr(), pdh, ldh, out.data_ptr(),
                         ldo)
    _enqueue("situ_moe_gated_backward", index, ctypes.byref(args))
    return out, h


class _ExpertFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w1, w2, offsets, p0, p1, activation, keep):
        gate_up = situ_moe_grouped_gemm(x, w1, offsets)
        h, q, scale = situ_moe_gated(gate_up, p0, p1, offsets, activation=activation, save=True)
        kept = (None, None) if not ctx.needs_input_grad[1] else situ_moe_save_mxfp8(x) if keep == "mxfp8" else (x, None)
        ctx.save_for_backward(*kept, q, scale, w1, w2, offsets, p0, p1)
        ctx.activation, ctx.dtype = activation, x.dtype
        return situ_moe_grouped_gemm(h, w2, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, x_scale, q, scale, w1, w2, offsets, p0, p1 = ctx.saved_tensors
        need_x, need_w1, need_w2 = ctx.needs_input_grad[:3]
        dx = dw1 = dw2 = None
        dh = situ_moe_grouped_gemm_dgrad(dy, w2, offsets)
        d, h = situ_moe_gated_backward(dh, q, scale, p0, p1, offsets, activation=ctx.activation, want_h=need_w2)
        if need_w2:
            dw2 = situ_moe_grouped_gemm_wgrad(dy, h, offsets)
        del dh, h
        if need_x:
            dx = situ_moe_grouped_gemm_dgrad(d, w1, offsets)
        if need_w1:
            dw1 = situ_moe_grouped_gemm_wgrad(d, x if x_scale is None else situ_moe_restore_mxfp8(x, x_scale, ctx.dtype),
                                              offsets)
        return dx, dw1, dw2, None, None, None, None, None


def expert_ffn(x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, offsets: torch.Tensor, p0: torch.Tensor,
               p1: torch.Tensor, *, activation: int = SITU_ACT_FN_SITU, keep: str = "mxfp8") -> torch.Tensor:
    """The routed experts for training: y = w2_e gated(w1_e x) over rows sorted by
    expert, differentiable in x [S, H], w1 [E, 2I, H] and w2 [E, H, I].  For the
    backward pass it keeps the gate/up columns in 8 bits, x in 8 bits
    (``keep`` "mxfp8") or as it is ("16bit"), and no h: 2 I + H bytes a row and
    a 32nd, where 16 bits take 6 I + 2 H.  p0 and p1 are constants."""
    if keep not in ("mxfp8", "16bit"):
        raise ValueError('keep must be "mxfp8" or "16bit"')
    if w1.dim() != 3 or w2.dim() != 3:
        raise ValueError("w1 must be [E, 2I, H] and w2 [E, H, I]")
    _constant(p0=p0, p1=p1)
    return _graphed(_ExpertFfn.apply, x, w1, w2, offsets, p0, p1, activation, keep)


def _adapters(x, a, b, scale, index):
    """Checks an adapter set beside x [S, K]: (a, b, their pointers, scale, S, K, N, r, n)."""
    dtype = x.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16 or a.dtype is not dtype or b.dtype is not dtype:
        raise TypeError("x, a and b must be all bf16 or all f16")
    try:
        (S, K), (n, r, Ka), (nb, N, rb) = x.shape, a.shape, b.shape
    except ValueError:
        raise ValueError("needs x [S, K], a [n, r, K] and b [n, N, r]") from None
    if Ka != K or nb != n or rb != r:
        raise ValueError(f"needs a [n, r, {K}] and b [n, N, r], not {tuple(a.shape)} and {tuple(b.shape)}")
    if (S | K | N | n) >> 31:
        raise _too_large(S, K, N, n)
    if index < 0 or a.get_device() != index or b.get_device() != index:
        raise ValueError(f"the operands must be on one CUDA device, not on {x.device}, {a.device} and {b.device}")
    if scale is not None:
        scale = _vector(scale, torch.float32, n, "scale", index)
    a, pa = _packed(a)
    b, pb = _packed(b)
    return a, b, pa, pb, scale, S, K, N, r, n


def _beside(t, shape, dtypes, name, index):
    """(tensor, pointer, elements between rows) of base or dx0."""
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must be {shape} of the operands' type or fp32, not {tuple(t.shape)} of {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} on {t.device}, the operands on cuda:{index}")
    return _rows(t, 4 if t.dtype is torch.float32 else 8)


def situ_moe_lora(base, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, *, ids=None, offsets=None, scale=None, out=None,
                  keep: bool = False, stream=None):
    """base + scale[e] (x a[e].T) b[e].T row by row: base [S, N] the shared
    projection of x [S, K] (None: zeros, of x's type), a [n, r, K] and b
    [n, N, r], e = ids[i] (int32 [S]; outside [0, n): no adapter) or the one
    whose rows ``offsets`` [n + 1] bounds.  ``out`` may be base.  ``keep``
    returns (out, u [S, 2, r], rounded and what that leaves) for
    situ_moe_lora_backward."""
    if stream is not None:
        return _on_stream(stream, lambda x, a, b, base, **kw: situ_moe_lora(base, x, a, b, **kw), x, a, b, base, ids=ids,
                          offsets=offsets, scale=scale, out=out, keep=keep)
    index = x.get_device()
    a, b, pa, pb, scale, S, K, N, r, n = _adapters(x, a, b, scale, index)
    if (ids is None) == (offsets is None):
        raise ValueError("needs one of ids and offsets")
    dtype, pids, poff = x.dtype, None, None
    if ids is not None:
        ids = _vector(ids, torch.int32, S, "ids", index)
        pids = ids.data_ptr()
    else:
        if _groups(offsets, index) != n:
            raise ValueError(f"offsets must be [{n + 1}]")
        if not offsets.is_contiguous():
            offsets = offsets.contiguous()
        poff = offsets.data_ptr()
    x, px, ldx = _rows(x, 8)
    pbase, ld_base, out_dtype = None, 0, dtype if out is None else out.dtype
    if base is not None:
        base, pbase, ld_base = _beside(base, (S, N), (dtype, torch.float32), "base", index)
        out_dtype = base.dtype
    new = _new(index)
    if out is None:
        out, ldo = new((S, N), (N, 1), out_dtype), N
    else:
        ldo = _given(out, (S, N), out_dtype, index, 4 if out_dtype is torch.float32 else 8)
    u = new((S, 2, r), (2 * r, r, 1), dtype) if keep else None
    size = _lora_bytes(S, K, N, r, n, index)
    ws, pws = _scratch(size, new)
    args = SituLoraArgs(_DTYPES[dtype], _DTYPES.get(out_dtype, -1), S, K, N, r, n, px, ldx, pa, pb, pids, poff,
                        None if scale is None else scale.data_ptr(), pbase, ld_base, out.data_ptr(), ldo,
                        None if u is None else u.data_ptr(), _status_word(index).data_ptr())
    _enqueue("situ_moe_lora", index, ctypes.byref(args), pws, size)
    return (out, u) if keep else out


def situ_moe_lora_backward(dy: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor,
                           u: torch.Tensor, *, scale=None, dx=None, out=None, dy_scale=None, stream=None):
    """The gradients of situ_moe_lora with rows sorted by adapter, from dy [S, N]
    and its u: (dx [S, K], da, db).  ``dx`` is what x's gradient is added to
    (that of the shared projection; None: zeros, of x's type), and ``out``,
    which may be it, receives the sum.  dy counts times ``dy_scale``, one fp32 on
    the device."""
    if stream is not None:
        return _on_stream(stream, situ_moe_lora_backward, dy, x, a, b, offsets, u, scale=scale, dx=dx, out=out,
                          dy_scale=dy_scale)
    index = x.get_device()
    a, b, pa, pb, scale, S, K, N, r, n = _adapters(x, a, b, scale, index)
    dtype = x.dtype
    if dy.dtype is not dtype or u.dtype is not dtype:
        raise TypeError(f"dy and u must be {dtype}, as x")
    if dy.shape != (S, N) or u.shape != (S, 2, r):
        raise ValueError(f"needs dy {(S, N)} and u {(S, 2, r)}")
    _on_device(index, dy=dy, u=u)
    if _groups(offsets, index) != n:
        raise ValueError(f"offsets must be [{n + 1}]")
    if not offsets.is_contiguous():
        offsets = offsets.contiguous()
    x, px, ldx = _rows(x, 8)
    dy, pdy, ld_dy = _rows(dy, 8)
    u, pu = _packed(u)
    pdx0, ld_dx0, dx_dtype = None, 0, dtype if out is None else out.dtype
    if dx is not None:
        dx, pdx0, ld_dx0 = _beside(dx, (S, K), (dtype, torch.float32), "dx", index)
        dx_dtype = dx.dtype
    if dy_scale is not None and (dy_scale.dtype is not torch.float32 or dy_scale.numel() != 1
                                 or dy_scale.get_device() != index):
        raise ValueError(f"dy_scale must be one fp32 on cuda:{index}")
    new = _new(index)
    if out is None:
        out, ldo = new((S, K), (K, 1), dx_dtype), K
    else:
        ldo = _given(out, (S, K), dx_dtype, index, 4 if dx_dtype is torch.float32 else 8)
    da, db = new((n, r, K), (r * K, K, 1), dtype), new((n, N, r), (N * r, r, 1), dtype)
    size = _lora_backward_bytes(S, K, N, r, index)
    ws, pws = _scratch(size, new)
    args = SituLoraBackwardArgs(_DTYPES[dtype], _DTYPES.get(dx_dtype, -1), S, K, N, r, n, pdy, ld_dy, px, ldx, pa, pb,
                                offsets.data_ptr(), None if scale is None else scale.data_ptr(), pu, pdx0,
                                ld_dx0, out.data_ptr(), ldo, da.data_ptr(), db.data_ptr(), _status_word(index).data_ptr(),
                                None if dy_scale is None else dy_scale.data_ptr())
    _enqueue("situ_moe_lora_backward", index, ctypes.byref(args), pws, size)
    return out, da, db


def _into_f16(t: torch.Tensor):
    """(t times a power of two, as f16; that power's inverse): the largest
    magnitude in [2^14, 2^15), all on the device."""
    most = torch.linalg.vector_norm(t, float("inf"))
    e = torch.where(torch.isfinite(most), 15 - torch.frexp(most).exponent, 0).clamp(-126, 126).int()
    power, back = ((127 + e) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    return torch.mul(t, power, out=torch.empty(t.shape, dtype=torch.float16, device=t.device)), back


class _LoraLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, base, x, a, b, offsets, scale):
        y, u = situ_moe_lora(base, x, a, b, offsets=offsets, scale=scale, keep=True)
        ctx.save_for_backward(x, a, b, offsets, u, scale)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, a, b, offsets, u, scale = ctx.saved_tensors
        dx = da = db = None
        if any(ctx.needs_input_grad[1:4]):
            if dy.dtype is torch.float32 and x.dtype is torch.float16 and dy.numel():
                d, back = _into_f16(dy)
            else:
                d, back = dy.to(x.dtype), None
            dx, da, db = situ_moe_lora_backward(d, x, a, b, offsets, u, scale=scale, dy_scale=back)
        return dy if ctx.needs_input_grad[0] else None, dx, da, db, None, None


def lora_linear(base: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor,
                scale=None) -> torch.Tensor:
    """situ_moe_lora for training, rows sorted by adapter: differentiable in
    base, x, a and b (up to 1,024 adapters).  Beside an fp32 base the incoming
    gradient is rounded to the operands' type for those of x, a and b, in f16
    under a power of two of its largest magnitude; base's is as it came.
    ``scale`` is a constant."""
    if a.shape[0] > 1024:
        raise ValueError("the gradients take up to 1024 adapters")
    _constant(scale=scale)
    return _graphed(_LoraLinear.apply, base, x, a, b, offsets, scale)


class Layer:
    """Keeps the argument struct and a workspace for one workload, so that a
    forward call is a single C-ABI call (the bench times exactly this)."""

    def __init__(self, wl, out: Optional[torch.Tensor] = None, x_q=None, x_scale=None,
                 pack_scales: bool = True, fuse_combine: bool = False, activation: int = 0,
                 apply_topk_in_fc1: bool = False, h1_nvfp4: bool = False):
        self.wl = wl
        dev = wl.x_bf16.device
        self.out = out if out is not None else torch.empty((wl.T, wl.H), dtype=torch.bfloat16,
                                                           device=dev)
        kw = dict(T=wl.T, H=wl.H, I=wl.I, num_experts_total=wl.E_total,
                  num_local_experts=wl.E_loc, local_expert_offset=wl.off, top_k=wl.K,
                  act_dtype=wl.act, weight_dtype=wl.wt, topk_ids=wl.topk_ids,
                  topk_weights=wl.topk_weights, w1=wl.w1, w1_scale=wl.w1_scale, w2=wl.w2,
                  w2_scale=wl.w2_scale, gemm1_alpha=wl.gemm1_alpha, gemm1_beta=wl.gemm1_beta,
                  g1_alphas=wl.g1_alphas, g1_alphas_up=wl.g1_alphas_up, g2_alphas=wl.g2_alphas,
                  w1_gscale=wl.w1_gscale, w2_gscale=wl.w2_gscale, out=self.out)
        if wl.act == SITU_ACT_BF16:
            kw["hidden_states"] = wl.x_bf16
        elif wl.act == SITU_ACT_MXFP8:
            if x_q is None:
                x_q = torch.empty((wl.T, wl.H), dtype=torch.uint8, device=dev)
                x_scale = torch.empty((wl.T, wl.H // 32), dtype=torch.uint8, device=dev)
            self.x_q, self.x_scale = x_q, x_scale
            kw["hidden_states_q"], kw["hidden_states_scale"] = x_q, x_scale
        else:
            # NVFP4: quantised from the bf16 hidden states on the GPU in every call
            self.x_q = torch.empty((wl.T, wl.H // 2), dtype=torch.uint8, device=dev)
            self.x_scale = torch.empty((wl.T, wl.H // 16), dtype=torch.uint8, device=dev)
            self.x_gscale = torch.empty((wl.T,), dtype=torch.float32, device=dev)
            kw["hidden_states_q"], kw["hidden_states_scale"] = self.x_q, self.x_scale
            kw["hidden_states_gscale"] = self.x_gscale
        self._keep = kw
        self.args = make_args(**kw)
        self.args.fuse_combine = 1 if fuse_combine else 0
        self.args.activation = int(activation)
        self.args.apply_topk_in_fc1 = 1 if apply_topk_in_fc1 else 0
        self.args.h1_nvfp4 = 1 if h1_nvfp4 else 0
        # weight scales in the block-scaled GEMMs' layout, packed once per
        # weight set (as at weight-load time) when the shapes use it
        self.scales_packed = None
        np_ = situ_moe_packed_scales_size(self.args) if pack_scales else 0
        if np_ > 0:
            self.scales_packed = torch.empty(np_, dtype=torch.uint8, device=dev)
            situ_moe_pack_scales(self.args, self.scales_packed)
            self.args.scales_packed = self.scales_packed.data_ptr()
        n = situ_moe_workspace_size(self.args)
        self.workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)

    def launches(self) -> int:
        """Kernels one __call__ enqueues (the forward, plus the activation
        quantisation for MXFP8 and NVFP4 activations)."""
        return situ_moe_forward_launches(self.args) + (0 if self.wl.act == SITU_ACT_BF16 else 1)

    def _quant(self, stream):
        if self.wl.act == SITU_ACT_MXFP8:
            situ_moe_quant_mxfp8(self.wl.x_bf16, stream, out=(self.x_q, self.x_scale))
        elif self.wl.act == SITU_ACT_NVFP4:
            situ_moe_quant_nvfp4(self.wl.x_bf16, stream, out=(self.x_q, self.x_scale, self.x_gscale))

    def device_status(self, stream=None) -> int:
        """0 when every bounded device wait of the last call completed."""
        return situ_moe_device_status(self.args, self.workspace, stream)

    def profiled(self, events, quant_events=None, stream=None) -> torch.Tensor:
        """Like __call__, recording per-stage events (see situ_moe_forward_profiled);
        ``quant_events`` (start, end) bracket the activation quantisation."""
        if self.wl.act != SITU_ACT_BF16:
            if quant_events:
                quant_events[0].record(stream)
            self._quant(stream)
            if quant_events:
                quant_events[1].record(stream)
        situ_moe_forward_profiled(self.args, self.workspace, events, stream)
        return self.out

    def capture(self, warmup: bool = True):
        """A CUDA graph of one __call__ (the activation quantisation, if any,
        and the forward's kernels, with their programmatic dependencies).
        situ_moe_forward never synchronises the host, so a call can be
        captured; the graph replays on the same buffers.  Returns the
        torch.cuda.CUDAGraph; ``graph.replay()`` runs one layer pass."""
        if warmup:   # one eager call first: per-device attribute set-up
            self()
            torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                self(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        return g

    def __call__(self, stream=None) -> torch.Tensor:
        """One pass of the layer; for MXFP8 and NVFP4 activations this includes
        their quantisation from the bf16 hidden states."""
        self._quant(stream)
        situ_moe_forward(self.args, self.workspace, stream)
        return self.out
