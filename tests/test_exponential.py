"""csrc/exponential.h on the host: every magnitude, both ends of float64 and beyond."""
from __future__ import annotations

import math
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "parameter_efficient_fine_dora_amd", "csrc")
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
using namespace std;
#define __device__
#define __forceinline__ inline
#include "exponential.h"

int main() {   // numbers from stdin; exp and exp - 1 of each
  char word[64];
  while (scanf("%63s", word) == 1) {
    const dora::Exponential e(strtod(word, nullptr));
    printf("%a %a\n", e.value(), e.less_one());
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def evaluate(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("exponential")
    (d / "e.cpp").write_text("#include <cmath>\n" + PROGRAM)
    res = subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, str(d / "e.cpp"), "-o", str(d / "e")],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]

    def run(values):
        out = subprocess.run([str(d / "e")], input="\n".join(map(repr, values)), capture_output=True,
                             text=True, timeout=60)
        assert out.returncode == 0
        return [tuple(float.fromhex(v) for v in line.split()) for line in out.stdout.splitlines()]

    return run


def test_the_ends(evaluate):
    """Infinite from float64's end on, and finite up to it, whichever side of a whole n log 2 a number
    lies; exp(d) - 1 too."""
    inf = math.inf
    big = [709.5, 709.78, 709.7827, 710.0, 745.0, 800.0, 800.3, 1000.0, 1000.3, 1099.9, 1100.0, 1e5, 1e300, inf]
    for x, (value, less) in zip(big, evaluate(big)):
        want = math.exp(x) if x < 709.7827128933841 else inf
        assert value == pytest.approx(want, rel=1e-12) and less == value, x
    small = [-v for v in big]
    for x, (value, less) in zip(small, evaluate(small)):
        # below float64's normal range a result keeps an absolute rounding
        assert abs(value - math.exp(x)) <= 1e-12 * math.exp(x) + 2.0 ** -1074 and less == -1.0, x
    value, less = evaluate([math.nan])[0]
    assert math.isnan(value) and math.isnan(less)
