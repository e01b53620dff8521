"""The tiles into which the linear layers cut an expert's rows (csrc/tiles.h), compiled by the host's compiler: up to the largest
row count they cover the rows once, none is empty or wider than the kernel's tile, and the widths are whole steps."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST_ROWS = 2 ** 31 - 2 ** 16
KERNELS = [(64, 16), (64, 32), (128, 32), (256, 32)]  # widest tile, step

PROGRAM = """
#include <stdio.h>
#include "tiles.h"
int main() {
    int most, step, cols;
    while (scanf("%d %d %d", &most, &step, &cols) == 3) {
        const int n = moe::lin_tiles(cols, most);
        printf("%d %d\\n", n, step == 16 ? moe::lin_width<16>(cols, n) : moe::lin_width<32>(cols, n));
    }
}
"""


def test_tiles_cover_the_rows(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "tiles.cpp", tmp_path / "tiles"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I", os.path.join(ROOT, "sparse_moe_ffn_router_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    counts = sorted({c for b in (1, 16, 32, 48, 64, 96, 128, 256, 512, 1000, 4096, 65536, 2 ** 24, 2 ** 30, 2_114_000_000, 2_131_000_000, 2_139_128_000, MOST_ROWS)
                     for c in range(b - 3, b + 4) if 1 <= c <= MOST_ROWS} | set(range(1, 1100)))
    cases = [(most, step, c) for most, step in KERNELS for c in counts]
    out = subprocess.run([str(exe)], input="".join("%d %d %d\n" % c for c in cases), capture_output=True, text=True, check=True).stdout.split()
    for (most, step, cols), n, width in zip(cases, map(int, out[::2]), map(int, out[1::2]), strict=True):
        assert n == -(-cols // most), (most, step, cols)
        assert 0 < width <= most and width % step == 0, (most, step, cols, width)
        assert (n - 1) * width < cols <= n * width, (most, step, cols, width)
