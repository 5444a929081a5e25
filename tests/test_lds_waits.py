"""Kernels that write their own barriers, as compiled: no wave reaches a barrier with LDS accesses under
way.  Behind such a barrier another wave may fill, or read, the same place."""
from __future__ import annotations

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from parameter_efficient_fine_dora_amd import build

OWN_BARRIERS = ["gemm.hip", "gram.hip", "orthogonal.hip"]


def under_way(assembly):
    """(barriers, [(kernel, line, LDS accesses that may be under way at that barrier)])."""
    kernel, pending, barriers, found = None, 0, 0, []
    for number, line in enumerate(assembly.splitlines(), 1):
        label = re.match(r"(_Z\w+):", line)
        if label:
            kernel, pending = label.group(1), 0
        op = line.strip()
        if op.startswith("ds_"):
            pending += 1
        count = re.match(r"s_waitcnt\b.*lgkmcnt\((\d+)\)", op)
        if count:
            pending = min(pending, int(count.group(1)))
        if op.startswith("s_barrier"):
            barriers += 1
            if pending:
                found.append((kernel, number, pending))
    return barriers, found


def test_the_look_finds_what_it_should():
    read = "_Z1k:\n ds_read_b128 v[0:3], v4\n ds_read_b128 v[8:11], v4\n"
    assert under_way(read + " s_barrier\n") == (1, [("_Z1k", 4, 2)])
    assert under_way(read + " s_waitcnt lgkmcnt(1)\n s_barrier\n") == (1, [("_Z1k", 5, 1)])
    assert under_way(read + " s_waitcnt vmcnt(0)\n s_barrier\n")[1]
    assert under_way(read + " s_waitcnt vmcnt(0) lgkmcnt(0)\n s_barrier\n") == (1, [])
    assert under_way(read + " s_endpgm\n_Z1j:\n s_barrier\n") == (1, [])


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """The sources' assembly, compiled side by side (gemm.hip alone takes most of a minute)."""
    at = tmp_path_factory.mktemp("waits")

    def compiled(source):
        out = at / (source + ".s")
        subprocess.run([build.hipcc(), *build.compile_flags(), "--cuda-device-only", "-S",
                        os.path.join(build.CSRC, source), "-o", str(out)], check=True,
                       stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL, timeout=600)
        return out.read_text()

    try:
        with ThreadPoolExecutor(len(OWN_BARRIERS)) as pool:
            return dict(zip(OWN_BARRIERS, pool.map(compiled, OWN_BARRIERS)))
    except OSError:
        pytest.skip("hipcc not available")


@pytest.mark.parametrize("source", OWN_BARRIERS)
def test_no_lds_access_is_under_way_at_a_barrier(assembly, source):
    barriers, found = under_way(assembly[source])
    assert barriers > 0 and not found, found


def test_every_source_with_its_own_barrier_is_looked_at():
    own = [s for s in build.SOURCES if '"s_barrier"' in open(os.path.join(build.CSRC, s)).read()]
    assert set(OWN_BARRIERS) == set(own)
