"""Shared memory of the log probability kernels (csrc/logprobs_pick.h), on the
host: enough, and in few sizes, since each is a key of the occupancy that is
kept for all operators."""
import os
import shutil
import subprocess

import pytest

from row_reduction_norm_gb300 import build as B

PROGRAM = r"""
#include "logprobs_pick.h"
#include <cstdio>
#include <set>

int main() {
    std::set<size_t> sizes;
    long wrong = 0;
    for (int unit : {1024, 2048})                                 // logits of a unit: fp32, bf16
        for (int vocab = 1; vocab <= 1 << 20; vocab += vocab < 9000 ? 1 : 1000) {
            const int units = (vocab + unit - 1) / unit;
            for (int warps = 1; warps <= 8; warps *= 2) {
                if (warps < 8 && warps < units) continue;         // a warp a unit, up to eight
                const size_t got = rrn::lp_smem(units, 8 / warps);
                wrong += got < (size_t)units * 12 * (8 / warps) || got > 16 * 1024;
                sizes.insert(got);
            }
        }
    std::printf("%ld %zu\n", wrong, sizes.size());
    return 0;
}
"""


def test_shared_memory_is_enough_and_in_few_sizes(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not installed")
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-I", B.CSRC, str(src), "-o", str(exe)], check=True)
    wrong, sizes = (int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert wrong == 0 and sizes <= 3                              # of sixteen kernels each


def test_the_call_asks_for_that():
    with open(os.path.join(B.CSRC, "logprobs_api.cu"), encoding="utf-8") as f:
        text = f.read()
    assert "smem = rrn::lp_smem(p.units, rrn::kLpWarps / p.warps);" in text
