"""Shared memory of the gradient's kernels whose need follows from the width
(csrc/dropout_pick.h), on the host: enough, within a block's limit, and in few
sizes, since each is a key of the occupancy that is kept for all operators."""
import shutil
import subprocess

import pytest

from row_reduction_norm_gb300 import build as B

PROGRAM = r"""
#include "dropout_pick.h"
#include <cstdio>
#include <set>

int main() {
    std::set<size_t> single, loop;
    long wrong = 0;
    for (int64_t hidden = 1; hidden <= 65536; ++hidden) {
        const size_t mask = (hidden + 7) / 8;
        for (int dropout = 0; dropout < 2; ++dropout) {
            const size_t a = rrn::drop_scalar_smem(hidden, dropout), b = rrn::drop_loop_smem(hidden, false, dropout);
            wrong += a < (dropout ? 2 * mask : 0) || b < (dropout ? mask : 0) || b > 226 * 1024;
            if (hidden <= 8192) single.insert(a);
            loop.insert(b);
            if (hidden > 49152) continue;
            const size_t c = rrn::drop_loop_smem(hidden, true, dropout);
            wrong += c < hidden * 4 + (dropout ? mask : 0) || c > 226 * 1024;
            loop.insert(c);
        }
    }
    std::printf("%ld %zu %zu\n", wrong, single.size(), loop.size());
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
    wrong, single, loop = (int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                                          check=True).stdout.split())
    # six kernels of single elements a type and direction of dw, four two-pass ones a type
    assert wrong == 0 and single <= 3 and loop <= 24
