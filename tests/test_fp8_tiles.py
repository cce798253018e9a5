"""How the 8-bit pair kernel cuts rows into tiles, without a GPU: the rule's own source, compiled for the host."""
import os
import shutil
import subprocess

import pytest

import dense_tiled_gemm_fp16_gb300 as g

CSRC = os.path.join(os.path.dirname(g.LIB_PATH), "csrc")

PROGRAM = r"""
#include <cstdio>
#include "fp8_tiles.h"
int main()
{
    long long rows;
    int w;
    while (std::scanf("%lld %d", &rows, &w) == 2) {
        const int parts = fp8_dev::parts_of(static_cast<int>(rows), w);
        std::printf("%d %d\n", parts, fp8_dev::width_of(static_cast<int>(rows), parts));
    }
}
"""


def test_parts_and_widths_of_any_number_of_rows(tmp_path):
    """Up to the most rows a call may have, parts hold all rows and are as equal as multiples of 32 allow."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "tiles.cpp", tmp_path / "tiles"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True, capture_output=True)
    most = g.MAX_DIM
    sizes = [0, 1, 31, 32, 33, 255, 256, 257, 1000, 131072, 2 ** 24 + 1, 2 ** 30, most - 2 ** 26, most - 2 ** 23, most - 1, most]
    cases = [(rows, w) for rows in sizes for w in range(32, 257, 32)]
    text = "\n".join(f"{r} {w}" for r, w in cases)
    out = subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout.split()
    got = list(zip(map(int, out[::2]), map(int, out[1::2])))
    for (rows, w), (parts, width) in zip(cases, got):
        assert parts == -(-rows // w)
        assert width == (-(-rows // parts) + 31) // 32 * 32 if rows else width == 0
        assert parts * width >= rows and width <= w
    assert len(got) == len(cases)
