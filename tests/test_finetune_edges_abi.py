"""Refusals of the fine-tuning operators' entry points that came later (no GPU needed)."""
import os
import re

import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build
from test_finetune_abi import lib, lora_back  # noqa: F401


@pytest.mark.parametrize("over,status", [(dict(dy_scale=0xb002), 6), (dict(dy_scale=0xb001, S=0), 6)])
def test_dy_scale_refusals(lib, over, status):  # noqa: F811
    assert lora_back(lib, **over) == status


def test_constants_that_ask_for_a_gradient_are_refused():
    # None came back for them without a word
    h, ad, off = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16), torch.tensor([0, 4, 4])
    one, leaf = torch.ones(2), torch.ones(2, requires_grad=True)
    for name, call in (("p0", lambda: B.expert_ffn(h, ad, ad, off, leaf, one)), ("p1", lambda: B.expert_ffn(h, ad, ad, off, one, leaf)),
                       ("scale", lambda: B.lora_linear(h, h, ad, ad, off, leaf))):
        with pytest.raises(ValueError, match=name + " gets no gradient"):
            call()
        with torch.no_grad(), pytest.raises((TypeError, ValueError)) as e:   # goes on to the devices' check
            call()
        assert "gradient" not in str(e.value)


def test_the_routers_grids_follow_the_devices_sm_count():
    # a constant of 152 put a second wave on a GPU of 148
    text = re.sub(r"//.*", "", open(os.path.join(build.CSRC, "balance.cu")).read())
    assert "sm_count()" in text and not re.search(r"kSms\s*=", text)


def test_the_router_needs_a_workspace_without_a_device_too(lib):  # noqa: F811
    assert lib.situ_moe_balance_loss_workspace_size(65536, 896) >= 152 * (2 * 896 + 1) * 4
