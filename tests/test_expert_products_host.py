"""What the expert products' kernels decide in plain arithmetic, compiled for
the host and run on the CPU."""
import ctypes
import os
import random
import re
import subprocess
import sys

import pytest
import torch

from block_scaled_fp4_permute_gb300 import binding as B, build

ROWS = r"""
#include <cstdio>
#include <vector>
#include "gemm_groups.cuh"
int main() {
  int S, E;
  while (scanf("%d %d", &S, &E) == 2) {
    std::vector<int32_t> off(E + 1);
    for (auto& o : off) scanf("%d", &o);
    bool asc = true;
    for (int e = 0; e < E; ++e) asc = asc && situ::gg::offset_at(off.data(), e, S) <= situ::gg::offset_at(off.data(), e + 1, S);
    for (int e = 0; e < E; ++e) {
      const int2 g = situ::gg::group_rows(off.data(), e, S, asc);
      printf("%d %d ", g.x, g.y);
    }
    printf("\n");
  }
}
"""


def run(tmp_path, source, text):
    src, exe = tmp_path / "host.cu", tmp_path / "host"
    src.write_text(source)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC, "-I",
                    os.path.join(build.ROOT, "include"), "-o", str(exe), str(src)], check=True, capture_output=True)
    return subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout


def test_groups_are_disjoint_whatever_the_offsets_hold(tmp_path):
    rng = random.Random(1)
    cases = [(50, [0, 10, 5, 2000000000, 60]), (50, [50, 0, 50, 0, 50, 0]), (7, [-3, -2147483648, 2147483647]), (0, [0, 5, 0]),
             (100, [0, 30, 30, 31, 100]), (1 << 30, [0, 1 << 30, 0, 1 << 30, 0, 2147483647])]
    for _ in range(300):
        S, E = rng.randrange(0, 60), rng.randrange(1, 9)
        off = [rng.randrange(-10, 70) for _ in range(E + 1)]
        cases.append((S, sorted(off) if rng.random() < 0.3 else off))
    text = "".join(f"{S} {len(off) - 1} {' '.join(map(str, off))}\n" for S, off in cases)
    lines = run(tmp_path, ROWS, text).splitlines()
    assert len(lines) == len(cases)
    for (S, off), line in zip(cases, lines):
        v = list(map(int, line.split()))
        at = [min(max(o, 0), S) for o in off]
        bound = [max(at[:i + 1]) for i in range(len(at))]
        assert v == [x for e in range(len(off) - 1) for x in (bound[e], bound[e + 1] - bound[e])]

LEAVE = r"""
#include <cstdio>
#include "gemm_groups.cuh"
int main() {
  // steps through a ring of three, whether the warp got through, the stage whose last arrival fails (-1: none)
  int steps, ok, fails;
  while (scanf("%d %d %d", &steps, &ok, &fails) == 3) {
    situ::gg::Ring<3> r;
    for (int i = 0; i < steps; ++i) r.next();
    auto arrived = [&](int j, uint32_t ph) {
      printf("a%d%u ", j, ph);
      return j != fails;
    };
    auto drain = [&] {
      situ::gg::last_uses(r, [&](int j, uint32_t ph) {
        printf("d%d%u ", j, ph);
        return false;
      });
    };
    situ::gg::leave(ok != 0, [&] { return situ::gg::last_uses(r, arrived); }, drain);
    printf("\n");
    situ::gg::leave(ok != 0, [&] { return situ::gg::last_use(r, arrived); }, drain);
    printf("\n");
  }
}
"""


def test_a_warp_drains_what_it_has_in_flight_unless_all_of_it_arrived(tmp_path):
    cases = [(steps, ok, fails) for steps in range(9) for ok in (0, 1) for fails in range(-1, 3)]
    lines = run(tmp_path, LEAVE, "".join("%d %d %d\n" % c for c in cases)).split("\n")
    for (steps, ok, fails), every, newest in zip(cases, lines[0::2], lines[1::2]):
        last = {i % 3: i // 3 % 2 for i in range(steps)}       # stage: parity of its last use
        drained = [f"d{j}{last[j]}" for j in sorted(last)]
        arrived = [f"a{j}{last[j]}" for j in sorted(last)] if ok else []
        assert every.split() == arrived + (drained if not ok or fails in last else []), (steps, ok, fails)
        j = (steps - 1) % 3
        arrived = [f"a{j}{last[j]}"] if ok and steps else []
        assert newest.split() == arrived + (drained if not ok or (steps and fails == j) else []), (steps, ok, fails)


def test_sizes_past_31_bits_are_refused_not_cut():
    # expanded tensors: one row of memory
    S = 2 ** 32 + 8
    off = torch.tensor([0, 4], dtype=torch.int32)

    def rows(n, dtype=torch.bfloat16):
        return torch.zeros(1, n, dtype=dtype).expand(S, n)

    w, wq = torch.zeros(1, 64, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.uint8)
    calls = [lambda: B.situ_moe_grouped_gemm(rows(64), w, off), lambda: B.situ_moe_grouped_gemm_dgrad(rows(64), w, off),
             lambda: B.situ_moe_grouped_gemm_wgrad(rows(64), rows(64), off),
             lambda: B.situ_moe_grouped_gemm_wgrad(rows(8)[:8], rows(8)[:8], off[:1].expand(S)),
             lambda: B.situ_moe_grouped_gemm(rows(64)[:4], rows(64)[None], off),
             lambda: B.situ_moe_quant_fp8(rows(64)), lambda: B.situ_moe_quant_fp8(rows(64)[None], 128),
             lambda: B.situ_moe_fp8_gemm(rows(64, torch.uint8), rows(1, torch.float32), wq, torch.zeros(1, 1)),
             lambda: B.situ_moe_fp8_gemm(wq, torch.zeros(64, 1), rows(64, torch.uint8), rows(1, torch.float32))]
    for call in calls:
        with pytest.raises(ValueError, match=r"below 2\^31"):
            call()


@pytest.mark.parametrize("over", [dict(lda=1 << 62), dict(ldo=1 << 62), dict(ldw=1 << 40), dict(direction=2, lda=64, ldb=1 << 62)])
def test_strides_beyond_the_tensor_maps_are_refused_by_their_size(over):
    build.build()
    a = dict(direction=0, dtype=0, out_dtype=0, S=16, N=64, K=128, E=4, accumulate=0, keep_rest=0, a=0x1000, lda=128,
             b=0x2000, ldb=128, offsets=0x3000, out=0x4000, ldo=64, device_status=0x5000)
    a.update(over)
    assert B.lib().situ_moe_grouped_gemm(ctypes.byref(B.SituGroupedGemmArgs(**a)), None) == 2


@pytest.mark.parametrize("over", [dict(ldx=1 << 62), dict(ldo=1 << 62), dict(ldw=1 << 40)])
def test_fp8_strides_beyond_the_tensor_maps_are_refused_by_their_size(over):
    build.build()
    a = dict(out_dtype=0, S=16, N=64, K=128, E=1, keep_rest=0, x_q=0x1000, ldx=128, x_scale=0x2000, w_q=0x3000,
             w_scale=0x4000, offsets=None, out=0x5000, ldo=64, device_status=0x6000)
    a.update(over)
    assert B.lib().situ_moe_fp8_gemm(ctypes.byref(B.SituFp8GemmArgs(**a)), None) == 2


def test_a_torch_without_the_direct_calls_takes_the_public_ones():
    # such as one built without CUDA
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name):\n"
            "        delattr(torch._C, name)\n"
            "from block_scaled_fp4_permute_gb300 import binding as B\n"
            "assert B._current_device is torch.cuda.current_device\n"
            "torch.cuda.current_stream = lambda index: type('S', (), {'cuda_stream': 7 + index})\n"
            "assert B._raw_stream(1) == 8\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=build.ROOT)


def test_kernels_that_share_registers_out_have_enough():
    build.build()
    for name, kernels in (("fp8_gemm", 3), ("grouped_gemm", 13)):
        with open(os.path.join(build.BUILD, name + ".cu.ptxas")) as f:
            log = f.read()
        names = re.findall(r"Compiling entry function '(\S+)'", log)
        assert sum(build._SHARING.search(n) is not None for n in names) == kernels
        assert build.short_of_registers(log) == []
    entry = "ptxas info    : Compiling entry function '_ZN4situ{}' for 'sm_103a'\n    0 bytes stack frame\nptxas info    : Used {} registers\n"
    log = entry.format("10f8w_kernelILi2ELi2EEEv", 160) + entry.format("9f8_kernelILi32ELb0EEEv", 40) + \
        entry.format("9gg_kernelILi2ELi0ELi256ELi1ELb0EEEv", 168) + entry.format("9gg_kernelILi2ELi0ELi256ELi2ELb0EEEv", 167) + \
        entry.format("9gg_kernelILi2ELi0ELi256ELi0ELb0EEEv", 72)
    assert [regs for _, regs in build.short_of_registers(log)] == [160, 167]
