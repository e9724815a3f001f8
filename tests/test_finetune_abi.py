"""Host-side checks of the fine-tuning operators' entry points (no GPU needed):
bad arguments are refused before anything is launched, and the binding's
structures have the header's layout."""
import ctypes
import os
import subprocess

import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


STRUCTS = {"situ_balance_args": B.SituBalanceArgs, "situ_router_backward_args": B.SituRouterBackwardArgs,
           "situ_gated_args": B.SituGatedArgs, "situ_lora_args": B.SituLoraArgs,
           "situ_lora_backward_args": B.SituLoraBackwardArgs}


def test_structures_have_the_headers_layout(tmp_path):
    lines = []
    for name, s in STRUCTS.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f[0]}));' for f in s._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include "situ_moe.h"\nint main(void) {' + "\n".join(lines) + " return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(build.ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    want = []
    for s in STRUCTS.values():
        want += [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def balance(lib, ws=0x9000, nbytes=1 << 30, **over):
    a = dict(router_logits=0x1000, ld=8, topk_ids=0x2000, mask=None, T=16, num_experts_total=8, top_k=2, coef=1.0,
             loss=0x3000, counts=0x4000, tokens=0x5000, row_stats=0x6000)
    a.update(over)
    return lib.situ_moe_balance_loss(ctypes.byref(B.SituBalanceArgs(**a)), ws, nbytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 2), (dict(num_experts_total=0), 2), (dict(num_experts_total=4097, ld=4097), 2), (dict(top_k=0), 2),
    (dict(top_k=9), 2), (dict(top_k=17, num_experts_total=64, ld=64), 2), (dict(ld=7), 2), (dict(ld=1 << 40), 2),
    (dict(router_logits=None), 1), (dict(topk_ids=None), 1), (dict(loss=None), 1), (dict(counts=None), 1),
    (dict(tokens=None), 1), (dict(row_stats=None), 1), (dict(T=4000, ws=None), 1), (dict(T=0, loss=None), 1),
    (dict(router_logits=0x1002), 6), (dict(row_stats=0x6004), 6), (dict(ws=0x9008), 6), (dict(counts=0x4001), 6),
    (dict(T=4000, nbytes=16), 4),
])
def test_balance_refusals(lib, over, status):
    assert balance(lib, **over) == status


def router_back(lib, **over):
    a = dict(router_logits=0x1000, ld=8, topk_ids=0x2000, mask=None, T=16, num_experts_total=8, top_k=2, renormalize=1,
             coef=1.0, counts=0x4000, tokens=0x5000, row_stats=0x6000, dloss=0x7000, topk_weights=0x8000, dweights=0x9000,
             dlogits=0xa000, ldo=8)
    a.update(over)
    return lib.situ_moe_router_backward(ctypes.byref(B.SituRouterBackwardArgs(**a)), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 2), (dict(num_experts_total=5000, ld=5000, ldo=5000), 2), (dict(top_k=9), 2), (dict(ld=4), 2),
    (dict(ldo=4), 2), (dict(renormalize=2), 3), (dict(counts=None), 1), (dict(tokens=None), 1), (dict(row_stats=None), 1),
    (dict(topk_weights=None), 1), (dict(topk_ids=None), 1), (dict(dlogits=None), 1), (dict(dlogits=0xa001), 6),
    (dict(row_stats=0x6004), 6), (dict(T=0, router_logits=None, dlogits=None), 0),
])
def test_router_backward_refusals(lib, over, status):
    assert router_back(lib, **over) == status


def gated(lib, back=False, **over):
    a = dict(dtype=0, activation=0, S=16, I=64, E=4, gate_up=0x1000, ld_gate_up=128, p0=0x2000, p1=0x3000, offsets=0x4000,
             h=0x5000, ldh=64, q=0x6000, scale=0x7000, dh=0x8000, ld_dh=64, dgate_up=0x9000, ld_dgate_up=128)
    a.update(over)
    return (lib.situ_moe_gated_backward if back else lib.situ_moe_gated)(ctypes.byref(B.SituGatedArgs(**a)), None)


@pytest.mark.parametrize("back,over,status", [
    (False, dict(dtype=2), 3), (False, dict(activation=2), 3), (True, dict(dtype=-1), 3), (False, dict(S=-1), 2),
    (False, dict(I=4), 2), (False, dict(I=60), 2), (True, dict(I=0), 2), (False, dict(E=0), 2), (False, dict(E=4097), 2),
    (False, dict(offsets=None), 2), (False, dict(ld_gate_up=120), 2), (False, dict(ld_gate_up=132), 2),
    (False, dict(ldh=56), 2), (True, dict(ld_dh=68), 2), (True, dict(ld_dgate_up=64), 2), (True, dict(ldh=8), 2),
    (False, dict(S=(1 << 30) + 1), 2), (False, dict(gate_up=None), 1), (False, dict(p0=None), 1), (False, dict(h=None), 1),
    (False, dict(q=None), 1), (False, dict(scale=None), 1), (True, dict(q=None), 1), (True, dict(scale=None), 1),
    (True, dict(dh=None), 1), (True, dict(dgate_up=None), 1), (False, dict(gate_up=0x1008), 6), (False, dict(q=0x6004), 6),
    (True, dict(dh=0x8008), 6), (True, dict(h=0x5008), 6), (False, dict(offsets=0x4002), 6),
    (False, dict(S=0, gate_up=None), 0), (True, dict(S=0, dh=None), 0),
])
def test_gated_refusals(lib, back, over, status):
    assert gated(lib, back, **over) == status


@pytest.mark.parametrize("args,status", [
    ((0x1000, 2, 4, 64, 64, 0x2000, 0x3000), 3), ((0x1000, 0, -1, 64, 64, 0x2000, 0x3000), 2),
    ((0x1000, 0, 4, 60, 64, 0x2000, 0x3000), 2), ((0x1000, 0, 4, 64, 56, 0x2000, 0x3000), 2),
    ((0x1000, 0, 4, 64, 68, 0x2000, 0x3000), 2), ((None, 0, 4, 64, 64, 0x2000, 0x3000), 1),
    ((0x1000, 0, 4, 64, 64, None, 0x3000), 1), ((0x1000, 0, 4, 64, 64, 0x2000, None), 1),
    ((0x1008, 0, 4, 64, 64, 0x2000, 0x3000), 6), ((0x1000, 0, 4, 64, 64, 0x2004, 0x3000), 6),
    ((None, 0, 0, 64, 64, None, None), 0),
])
def test_save_refusals(lib, args, status):
    assert lib.situ_moe_save_mxfp8(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((0x2000, 0x3000, 3, 4, 64, 0x1000, 64), 3), ((0x2000, 0x3000, 0, 4, 4, 0x1000, 64), 2),
    ((0x2000, 0x3000, 2, 4, 64, 0x1000, 66), 2), ((None, 0x3000, 0, 4, 64, 0x1000, 64), 1),
    ((0x2000, 0x3000, 0, 4, 64, None, 64), 1), ((0x2000, 0x3000, 0, 4, 64, 0x1008, 64), 6),
    ((None, None, 0, 0, 64, None, 64), 0),
])
def test_restore_refusals(lib, args, status):
    assert lib.situ_moe_restore_mxfp8(*args, None) == status


def lora(lib, ws=0xf000, nbytes=1 << 30, **over):
    a = dict(dtype=0, out_dtype=0, S=2000, K=64, N=128, r=16, n=4, x=0x1000, ldx=64, a=0x2000, b=0x3000, ids=0x4000,
             offsets=None, scale=None, base=0x5000, ld_base=128, out=0x6000, ldo=128, u=None, device_status=0xd000)
    a.update(over)
    return lib.situ_moe_lora(ctypes.byref(B.SituLoraArgs(**a)), ws, nbytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2, out_dtype=2), 3), (dict(out_dtype=1), 3), (dict(out_dtype=-1), 3), (dict(S=-1), 2), (dict(K=60), 2),
    (dict(K=0), 2), (dict(N=4), 2), (dict(r=0), 2), (dict(r=12), 2), (dict(r=136), 2), (dict(n=0), 2),
    (dict(n=(1 << 20) + 1), 2), (dict(ldx=56), 2), (dict(ldx=68), 2), (dict(ldo=120), 2), (dict(ld_base=64), 2),
    (dict(ld_base=132), 2), (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(out=None), 1),
    (dict(ids=None), 1), (dict(offsets=0x7000), 1), (dict(ws=None), 1), (dict(device_status=None), 1),
    (dict(device_status=0xd001), 6), (dict(x=0x1008), 6), (dict(a=0x2008), 6),
    (dict(b=0x3002), 6), (dict(base=0x5008), 6), (dict(out=0x6004), 6), (dict(u=0x8008), 6), (dict(ids=0x4001), 6),
    (dict(scale=0x9002), 6), (dict(ws=0xf008), 6), (dict(nbytes=16), 4), (dict(S=0, x=None), 0),
])
def test_lora_refusals(lib, over, status):
    assert lora(lib, **over) == status


def lora_back(lib, ws=0xf000, nbytes=1 << 30, **over):
    a = dict(dtype=0, dx_dtype=0, S=100, K=64, N=128, r=16, n=4, dy=0x1000, ld_dy=128, x=0x2000, ldx=64, a=0x3000,
             b=0x4000, offsets=0x5000, scale=None, u=0x6000, dx0=None, ld_dx0=0, dx=0x7000, ld_dx=64, da=0x8000, db=0x9000,
             device_status=0xa000)
    a.update(over)
    return lib.situ_moe_lora_backward(ctypes.byref(B.SituLoraBackwardArgs(**a)), ws, nbytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), 3), (dict(dx_dtype=1), 3), (dict(n=1025), 2), (dict(r=4), 2), (dict(ld_dy=64), 2), (dict(ld_dx=32), 2),
    (dict(dx0=0xb000), 2), (dict(dy=None), 1), (dict(x=None), 1), (dict(u=None), 1), (dict(dx=None), 1), (dict(da=None), 1),
    (dict(db=None), 1), (dict(offsets=None), 1), (dict(device_status=None), 1), (dict(ws=None), 1), (dict(dy=0x1008), 6),
    (dict(u=0x6008), 6), (dict(db=0x9008), 6), (dict(offsets=0x5002), 6), (dict(nbytes=64), 4),
])
def test_lora_backward_refusals(lib, over, status):
    assert lora_back(lib, **over) == status


def test_null_args_and_sizes(lib):
    for f in (lib.situ_moe_balance_loss, lib.situ_moe_lora, lib.situ_moe_lora_backward):
        assert f(None, 0x1000, 1 << 20, None) == 1
    for f in (lib.situ_moe_router_backward, lib.situ_moe_gated, lib.situ_moe_gated_backward):
        assert f(None, None) == 1
    assert lib.situ_moe_balance_loss_workspace_size(-1, 8) == 0 and lib.situ_moe_balance_loss_workspace_size(8, 5000) == 0
    assert lib.situ_moe_lora_workspace_size(8, 64, 64, 12, 1) == 0 and lib.situ_moe_lora_backward_workspace_size(8, 60, 64, 8) == 0
    assert lib.situ_moe_balance_loss_workspace_size(4000, 8) > 0 and lib.situ_moe_lora_workspace_size(1000, 64, 64, 8, 1) > 0
    # few tokens or rows take none
    assert lib.situ_moe_balance_loss_workspace_size(10, 8) == 0 and lib.situ_moe_lora_workspace_size(8, 64, 64, 8, 1) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    f, h = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.bfloat16)
    ids, one = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(1)
    u8 = torch.zeros(4, 8, dtype=torch.uint8)
    ad = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    off = torch.tensor([0, 4, 4], dtype=torch.int32)
    stats = torch.zeros(4, 2)
    for call in (lambda: B.situ_moe_balance_loss(f, ids), lambda: B.situ_moe_router_backward(f, ids, None, None, stats),
                 lambda: B.situ_moe_save_mxfp8(h), lambda: B.situ_moe_restore_mxfp8(u8, u8[:, :1]),
                 lambda: B.situ_moe_gated(h, one, one), lambda: B.situ_moe_gated_backward(h[:, :4], u8, u8[:, :2], one, one),
                 lambda: B.situ_moe_lora(None, h, ad, ad, offsets=off),
                 lambda: B.situ_moe_lora_backward(h, h, ad, ad, off, h[:, None])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: B.situ_moe_balance_loss(h, ids), lambda: B.situ_moe_balance_loss(f, ids.long()),
                 lambda: B.situ_moe_save_mxfp8(f), lambda: B.situ_moe_restore_mxfp8(u8, u8[:, :1], torch.float64),
                 lambda: B.situ_moe_gated(f, one, one), lambda: B.situ_moe_gated_backward(f, u8, u8[:, :2], one, one),
                 lambda: B.situ_moe_lora(None, f, ad, ad, offsets=off), lambda: B.situ_moe_lora(None, h, ad.half(), ad, offsets=off)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="keep"):
        B.expert_ffn(h, ad, ad, off, one, one, keep="8bit")


def test_sizes_past_31_bits_are_refused_not_cut():
    S = 2 ** 32 + 8
    rows = torch.zeros(1, 8, dtype=torch.bfloat16).expand(S, 8)
    bytes_ = torch.zeros(1, 8, dtype=torch.uint8).expand(S, 8)
    for call in (lambda: B._router(torch.zeros(1, 8).expand(S, 8), torch.zeros(1, 2, dtype=torch.int32).expand(S, 2), None),):
        with pytest.raises(ValueError):
            call()
    ad = torch.zeros(1, 8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=r"below 2\^31"):
        B._adapters(rows, ad, ad, None, 0)
    for call in (lambda: B.situ_moe_save_mxfp8(rows), lambda: B.situ_moe_restore_mxfp8(bytes_, bytes_[:, :1])):
        with pytest.raises(ValueError):
            call()
