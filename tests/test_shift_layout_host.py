"""How rows of odd widths lie on 16-byte chunks (csrc/shift_layout.h), checked
on the host: every chunk that the kernels take whole lies within the tensor,
and the rows' own elements cover it once each."""
import os
import shutil
import subprocess

import pytest

from row_reduction_norm_gb300 import build as B

PROGRAM = r"""
#include "shift_layout.h"
#include <cstdio>
#include <initializer_list>

template <int V>
long check(long hidden, long rows, long first) {
    long wrong = 0;
    for (long row = first; row < rows; ++row) {
        rrn::ShiftedRow<V> at;
        at.set(row, hidden);
        const long start = row * hidden - at.s;   // of chunk 0
        long own = 0;
        if (start < 0 || start % V != 0) ++wrong;
        for (int u = 0; u < at.chunks; ++u) {
            if (start + u * V + at.lo(u) != row * hidden + own) ++wrong;   // the row's next element
            own += at.hi(u) - at.lo(u);
            if (at.whole(u, row, rows, hidden) && start + (u + 1) * V > rows * hidden) ++wrong;   // read past the end
            if (at.whole(u, row, rows, hidden) != (start + (u + 1) * V <= rows * hidden)) ++wrong;
        }
        if (own != hidden) ++wrong;
    }
    return wrong;
}

int main() {
    for (long hidden = 1; hidden <= 40; ++hidden)
        for (long rows = 1; rows <= 4120; rows += rows < 20 || rows >= 4094 ? 1 : 407) {
            const long a = check<8>(hidden, rows, rows > 24 ? rows - 24 : 0);
            const long b = check<4>(hidden, rows, rows > 24 ? rows - 24 : 0);
            if (a || b) std::printf("%ld columns, %ld rows: %ld wrong of 8 a chunk, %ld of 4\n", hidden, rows, a, b);
        }
    for (long hidden : {101L, 1001L, 2047L, 8191L, 16379L})
        if (check<8>(hidden, 4100, 4080) || check<4>(hidden, 4100, 4080)) std::printf("%ld columns\n", hidden);
    return 0;
}
"""


def test_whole_chunks_lie_within_the_tensor(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not installed")
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", B.CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out == "", out[:2000]
