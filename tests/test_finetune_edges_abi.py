"""Refusals of the fine-tuning operators' entry points that came later (no GPU needed)."""
import pytest

from test_finetune_abi import lib, lora_back  # noqa: F401


@pytest.mark.parametrize("over,status", [(dict(dy_scale=0xb002), 6), (dict(dy_scale=0xb001, S=0), 6)])
def test_dy_scale_refusals(lib, over, status):  # noqa: F811
    assert lora_back(lib, **over) == status
