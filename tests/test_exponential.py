"""csrc/exponential.h on the host: every magnitude, both ends of float64 and beyond."""
from __future__ import annotations

import math
import os
import shutil
import subprocess
from decimal import Decimal, localcontext

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


def test_numbers_between(evaluate):
    """float64's own precision.  With |r| <= 0.3466 and q in [-0.293, 0.414]: q is off by its rounding, 2^-55,
    by r's, 2^-55, and by the sum's, a fifth of it twice rounded, 2^-56; 1 + q by 2^-53 of itself more, in all
    under 2^-52.  2^n q + (2^n - 1) raises q's 2^-54 to at most 2 2^-54 / 0.414 (n = 1) and rounds once: under
    2^-51.  (One log 2 of float64 instead of two parts is 2^-57 n off: 1e-14 at 700; sums to r^10 are 2e-13.)"""
    xs = [0.0, 1e-300, 1e-17, 1e-9, 1e-3, 0.1, 0.34657, 0.34658, 0.396, 1.0, 1.0397, 10.0, 44.3, 45.1, 100.3, 417.605, 700.1]
    xs += [-x for x in xs]
    with localcontext() as c:
        c.prec = 400   # of 1 + 1e-300, and what is left of it without the 1
        for x, (value, less) in zip(xs, evaluate(xs)):
            exp = Decimal(x).exp()
            assert abs(Decimal(value) - exp) <= Decimal(2.0 ** -52) * exp, x
            assert abs(Decimal(less) - (exp - 1)) <= Decimal(2.0 ** -51) * abs(exp - 1), x
