"""The adapters' kernels begin before their predecessor has ended, and give a wait up
after 200 ms.  A wait for what comes of the predecessor's results therefore begins
after griddep_wait(): the predecessor may take longer than that.  Read from the
sources (no GPU needed): calls that make a predecessor run so long take 100 GB."""
import os
import re

import pytest

from block_scaled_fp4_permute_gb300 import build


def role(file, kernel, name):
    """The source of one role of a kernel's warps, without comments."""
    text = open(os.path.join(build.CSRC, file)).read()
    text = text[text.index(f"\n{kernel}("):]
    text = text[:text.index("\n}\n")]
    part = text.split(f"// ---------------- {name} ----------------")
    assert len(part) == 2, (kernel, name)
    return re.sub(r"//.*", "", part[1].split("// ----------------")[0])


@pytest.mark.parametrize("file,kernel,name,wait", [
    ("lora.cu", "expand_kernel", "base in, out", "warp_wait(ydone"),
    ("lora.cu", "expand_kernel", "MMAs", "warp_wait(u_full"),
    ("lora.cu", "expand_kernel", "weights", "warp_wait(wempty"),
    ("lora_grads.cu", "outer_kernel", "MMAs", "warp_wait("),
    ("lora_grads.cu", "outer_kernel", "sums to memory, a column per lane", "warp_wait("),
])
def test_waits_for_the_predecessor_begin_after_it(file, kernel, name, wait):
    text = role(file, kernel, name)
    assert "griddep_wait()" in text and text.index("griddep_wait()") < text.index(wait)


def test_sums_wait_after_u_has_been_staged():
    # the epilogue's own waits follow the staging of u, whose second round begins with griddep_wait()
    text = open(os.path.join(build.CSRC, "lora.cu")).read()
    text = text[text.index("\nexpand_kernel("):]
    assert text.index("if (first && round == 1) griddep_wait();") < text.index("// ---------------- sums onto base")


def test_weights_leave_after_the_predecessor():
    text = role("lora.cu", "expand_kernel", "weights")
    assert "griddep_wait();" in text[:text.index("leave(")].splitlines()[-2]
