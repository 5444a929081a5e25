"""csrc/launch_cut.h on the host: every element of every tensor in exactly one piece, launches within
the threads that HIP takes, tensors up to the largest that the header allows."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "parameter_efficient_fine_dora_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "launch_cut.h"

// sizes...; prints a line per launch: workgroups and its pieces as tensor:at:n:block
int main(int argc, char** argv) {
  const int threads = atoi(argv[1]);
  const long chunk = atol(argv[2]);
  const int tensors = atoi(argv[3]);
  std::vector<int64_t> size;
  for (int i = 4; i < argc; ++i) size.push_back(atoll(argv[i]));
  std::vector<std::vector<int64_t>> pieces(tensors);
  const int rc = dora::cut_launches<int>(
      (int64_t)size.size(), chunk, tensors, dora::launch_blocks(threads),
      [&](int64_t i) { return size[i]; },
      [&](int k, int64_t i, int64_t at, int64_t n, int64_t block) { pieces[k] = {i, at, n, block}; },
      [&](int k, int64_t blocks) {
        printf("%lld", (long long)blocks);
        for (int j = 0; j < k; ++j)
          printf(" %lld:%lld:%lld:%lld", (long long)pieces[j][0], (long long)pieces[j][1],
                 (long long)pieces[j][2], (long long)pieces[j][3]);
        printf("\n");
        return 0;
      });
  return rc;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("cut")
    (d / "cut.cpp").write_text(PROGRAM)
    out = str(d / "cut")
    res = subprocess.run([gxx, "-std=c++17", "-O0", "-I", CSRC, str(d / "cut.cpp"), "-o", out],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-4000:]
    return out


MOST = (1 << 34) - 1      # elements of the largest tensor


@pytest.mark.parametrize("threads,chunk,tensors", [(512, 2048, 77), (256, 2048, 59), (256, 16384, 200)])
@pytest.mark.parametrize("sizes", [
    [MOST], [MOST - 2047], [MOST - 2046], [1 << 33], [(1 << 33) + 1], [(1 << 33) - 5, 7, MOST, 0, 3000],
    [1] * 500, [0], [0, 5, 0], [2048, 2049, 2047],
])
def test_every_element_once_and_launches_within_the_threads(program, threads, chunk, tensors, sizes):
    out = subprocess.run([program, str(threads), str(chunk), str(tensors), *map(str, sizes)],
                         capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    covered = [0] * len(sizes)
    for line in out.stdout.splitlines():
        blocks, *pieces = line.split()
        assert 0 < int(blocks) and int(blocks) * threads < 1 << 32
        assert 0 < len(pieces) <= tensors
        block = 0
        for piece in pieces:
            i, at, n, first = map(int, piece.split(":"))
            assert first == block and at == covered[i] and at % chunk == 0 and n > 0
            block += -(-n // chunk)
            covered[i] += n
        assert block == int(blocks)
    assert covered == sizes
