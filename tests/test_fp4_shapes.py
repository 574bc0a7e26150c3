"""The choice of workgroup shapes of the products with 4-bit weights (csrc/fp4_shape.h), compiled for the host: the
GPU tests take every shape, in every form, and the choice stays near the least estimated time."""

import os
import subprocess

import pytest

from fp8_fine_grained_amd import build
from tests.test_gpu_fp4 import SHAPED

SOURCE = """
#include <cstdio>
#include <cstdlib>
#include "fp4_shape.h"
using namespace fp8fg;
int main(int argc, char** argv) {
  printf("%d\\n", kFp4ShapeCount);
  for (int i = 1; i + 5 < argc; i += 6) {
    const int64_t M = atoll(argv[i]), N = atoll(argv[i + 1]), G = atoll(argv[i + 2]);
    const bool grouped = atoi(argv[i + 3]) != 0, gated = atoi(argv[i + 4]) != 0, codes = atoi(argv[i + 5]) != 0;
    printf("%d\\n", choose_fp4_shape(M, N, G, grouped, gated, codes, 256));
  }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    d = tmp_path_factory.mktemp("fp4_shape")
    (d / "c.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, str(d / "c.cpp"), "-o", str(d / "c")], check=True)

    def run(*problems):
        args = [str(int(v)) for p in problems for v in p]
        out = subprocess.run([os.path.join(d, "c"), *args], check=True, capture_output=True, text=True).stdout.split()
        return int(out[0]), [int(v) for v in out[1:]]
    return run


@pytest.mark.parametrize("codes", [False, True])
def test_the_gpu_tests_take_every_shape_in_every_form(choose, codes):
    for gated in (False, True):
        count, dense = choose(*[(M, N // 2 if gated else N, 1, False, gated, codes) for M, N in SHAPED])
        assert sorted(set(dense)) == list(range(count)), (gated, dense)
        # over two segments, one of them empty, the estimate halves the rows: other shapes, still most of them
        _, grouped = choose(*[(M, N // 2 if gated else N, 2, True, gated, codes) for M, N in SHAPED])
        assert len(set(grouped)) >= 8, (gated, grouped)


def test_choices(choose):
    _, got = choose((1, 4096, 1, False, False, False), (1, 2048, 1, False, True, False),
                    (5, 7168, 1, False, False, True), (8, 4096, 1, False, False, False), (16, 4096, 1, False, False, False),
                    (32, 7168, 1, False, False, True), (64, 7168, 1, False, False, False),
                    (128, 2048, 32, True, True, False), (8, 2048, 256, True, True, False))
    assert got == [0, 0, 4, 3, 6, 10, 11, 5, 2]
