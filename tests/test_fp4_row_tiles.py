"""Row tiles of the products with 4-bit weights (csrc/fp4_shape.h), compiled for the host: segments of up to 2^31 - 1
rows, where the rows and a tile's together pass 31 bits."""

import os
import subprocess

import pytest

from fp8_fine_grained_amd import build

SOURCE = """
#include <cstdio>
#include <cstdlib>
#include "fp4_shape.h"
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3)
    printf("%d\\n", fp8fg::fp4_row_tiles(atoi(argv[i]), atoi(argv[i + 1]), atoi(argv[i + 2])));
}
"""


@pytest.fixture(scope="module")
def row_tiles(tmp_path_factory):
    d = tmp_path_factory.mktemp("fp4_row_tiles")
    (d / "c.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, str(d / "c.cpp"), "-o", str(d / "c")], check=True)

    def run(*problems):
        args = [str(v) for p in problems for v in p]
        out = subprocess.run([os.path.join(d, "c"), *args], check=True, capture_output=True, text=True).stdout
        return [int(v) for v in out.split()]
    return run


@pytest.mark.parametrize("rows", [2, 8, 16, 32])
def test_row_tiles(row_tiles, rows):
    top = 2 ** 31 - 1
    problems = [(lo, hi, rows) for lo in (0, 1, 31, 32, 1000, top - 33, top - 1, top)
                for hi in (*range(lo, min(lo + 70, top + 1)), top - 65, top - 32, top - 31, top - 30, top - 1, top)
                if lo <= hi]
    assert row_tiles(*problems) == [-(-(hi - lo) // rows) for lo, hi, _ in problems]
