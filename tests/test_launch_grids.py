"""Grids that the host computes, compiled alone and run without a GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gradient_sync_ddp_gb300", "csrc")

PROGRAM = """
#include <cstdio>
#include <initializer_list>
#include "row_grid.h"
int main() {
    for (int wave = 1; wave <= 700; ++wave)
        for (long long need : {1ll, 2ll, 5ll, 7ll, 8ll, 9ll, 63ll, 151ll, 152ll, 153ll, 607ll, 608ll, 5000ll, 1ll << 40}) {
            const long long g = ddp::alike_grid(wave < need ? wave : static_cast<int>(need), need);
            const bool whole = g % 8 == 0 || g == need;
            if (g < 1 || g > need || g > (wave + 7) / 8 * 8 || !whole) {
                std::printf("wave %d need %lld: %lld\\n", wave, need, g);
                return 1;
            }
        }
    return 0;
}
"""


def test_grid_of_rows_that_lie_alike(tmp_path):
    """At least one CTA, never more than the work; a CTA takes either one piece or every grid-th with the grid a multiple
    of 8, on a GPU of any size."""
    if shutil.which("g++") is None:
        pytest.skip("needs a C++ compiler")
    src, exe = tmp_path / "grid.cpp", tmp_path / "grid"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True, capture_output=True,
                   text=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
