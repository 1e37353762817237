"""How long mla_key_weight's waits may take, on the CPU: longer than the work that they wait for, over all sizes that it takes."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_prologue_kv_gb300", "csrc")
PROGRAM = """
#include <stdio.h>
#include "key_weight_plan.cuh"
int main() {
    long long rows, keys;
    while (scanf("%lld %lld", &rows, &keys) == 2) printf("%d\\n", kvr::kw_patience(rows, keys));
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_waits_last_longer_than_a_tile_and_a_run(tmp_path):
    src, exe = tmp_path / "patience.cpp", tmp_path / "patience"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    sizes = [(r, k) for r in [1, 65536, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 45 << 20, 88 << 20, (1 << 30) - 5, (1 << 31) - 512]
             for k in (0, 1, 1 << 14, (1 << 22) - 1, 1 << 22, 1 << 24)]
    out = subprocess.run([str(exe)], input="".join("%d %d\n" % s for s in sizes), check=True, capture_output=True, text=True).stdout
    for (rows, keys), more in zip(sizes, map(int, out.split())):
        # all rows of a tile, at twice the 101 ns of the slowest ones, and all tiles of a run, at twice their 5 us
        assert 1 + more >= 2 * rows * 101e-9 and 1 + more >= 2 * keys / 256 * 5e-6
        assert rows >= 1 << 22 or keys >= 1 << 22 or more == 0   # ordinary calls: one second
