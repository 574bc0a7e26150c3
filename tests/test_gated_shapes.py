"""The sizes of the GPU tests take every workgroup shape that each form of the gated products
can choose.  The library's own rule is compiled and asked, so a change of it cannot drop a
shape out of the tests unseen.  Needs no GPU."""

import itertools
import os
import shutil
import subprocess

import pytest

from fp8_fine_grained_amd import build
from tests.gated_sizes import DENSE, EXPERTS

CUS = 256  # MI355X
SMALL, TILE128, TILE256 = set(range(6)), 6, 7

MAIN = r"""
#include <cstdio>
#include "gated_shape.h"
int main() {
  long long M, I, K, G;
  int grouped, exact, quantised, tiles_only;
  double cus;
  while (std::scanf("%lld %lld %lld %lld %d %d %d %d %lf", &M, &I, &K, &G, &grouped, &exact, &quantised, &tiles_only,
                    &cus) == 9)
    std::printf("%d\n", fp8fg::choose_gated_shape({M, I, K, G, grouped != 0, exact != 0, quantised != 0,
                                                   tiles_only != 0}, cus));
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/lib/llvm/bin/clang++"
    d = tmp_path_factory.mktemp("shape")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.CSRC, str(d / "main.cpp"), "-o", str(d / "main")], check=True)

    def ask(problems):
        """Shape index of each (M, I, K, G or 0, exact, quantised, tiles only)."""
        text = "".join(f"{M} {I} {K} {max(G, 1)} {int(G > 0)} {int(e)} {int(q)} {int(t)} {CUS}\n"
                       for M, I, K, G, e, q, t in problems)
        r = subprocess.run([str(d / "main")], input=text, capture_output=True, text=True, check=True)
        return [int(v) for v in r.stdout.split()]

    return ask


def _sizes(grouped):
    return [(sum(c), inner, K, len(c)) for c, inner, K in EXPERTS] if grouped else [(*s, 0) for s in DENSE]


@pytest.mark.parametrize("grouped,exact,quantised", itertools.product([False, True], repeat=3))
def test_every_shape_of_every_form_is_tested(choose, grouped, exact, quantised):
    got = choose([(*s, exact, quantised, False) for s in _sizes(grouped)])
    want = SMALL | {TILE128} | (set() if exact or grouped else {TILE256})
    assert set(got) == want, dict(zip(_sizes(grouped), got))
    # (the shape with several K blocks, so that its ring and its stages go round)
    assert {s for s, (_, _, K, _) in zip(got, _sizes(grouped)) if K >= 5 * 128} == want


def test_no_other_shape_is_ever_chosen(choose):
    rows = [1, 2, 7, 16, 17, 33, 64, 65, 128, 200, 300, 777, 1500, 4096, 8192]
    widths = [128, 384, 1152, 2048, 4096, 18432]
    for exact, quantised, tiles_only in itertools.product([False, True], repeat=3):
        dense = choose([(M, inner, K, 0, exact, quantised, tiles_only)
                        for M, inner, K in itertools.product(rows, widths, [128, 640, 2304, 7168])])
        experts = choose([(M, inner, K, G, exact, quantised, tiles_only)
                          for M, inner, K, G in itertools.product(rows, widths, [128, 2304, 7168], [1, 5, 32, 256])])
        least = TILE128 if tiles_only else 0
        assert set(dense) <= set(range(least, TILE256 if exact else TILE256 + 1))
        assert set(experts) <= set(range(least, TILE128 + 1))


def test_the_workspace_is_asked_for_where_a_small_shape_is_chosen(choose):
    """The library's own answer, on the same sizes (with no GPU it counts 256 units, as here)."""
    from fp8_fine_grained_amd import layer

    L = layer.lib()
    for grouped, exact in itertools.product([False, True], repeat=2):
        shapes = choose([(*s, exact, True, False) for s in _sizes(grouped)])
        for (M, inner, K, G), shape in zip(_sizes(grouped), shapes):
            want = 4 * M * inner if shape < TILE128 else 0
            assert L.fp8_block_gated_gemm_quant_workspace(1 if exact else 0, M, inner, K, G) == want
