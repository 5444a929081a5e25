"""Build libdora.so (HIP, gfx950) with hipcc and the compiled Python binding _bind.so with the
host compiler, both in-tree.

    python -m parameter_efficient_fine_dora_amd.build

Each source is compiled to an object in _build/ (in parallel), then linked
into parameter_efficient_fine_dora_amd/libdora.so next to the Python binding.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdora.so")
BIND = os.path.join(HERE, "_bind.so")   # csrc/bind.cpp
SOURCES = ["api.hip", "gemm.hip", "gram.hip", "rowwise.hip", "small.hip", "probe.hip", "noalloc.hip",
           "layernorm.hip", "logprob.hip", "adamw.hip", "preference.hip", "policy.hip",
           "orthogonal.hip"]
HEADERS = ["common.h", "kernels.h", "entry.h", "elem.h", "checks.h", "launch_cut.h", "sequences.h"]
ARCH = "gfx950"


def hipcc() -> str:
    env = os.environ.get("HIPCC")
    if env:
        return env
    found = shutil.which("hipcc")
    return found or "/opt/rocm/bin/hipcc"


def compile_flags() -> list[str]:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
        # packed-FP32 VALU forms are kept out of the generated code on purpose
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", os.path.join(ROOT, "include"), "-Wall", "-Wno-unused-function",
    ]


def bind_command(out: str) -> list[str]:
    """csrc/bind.cpp against torch's headers and libraries (which the process has loaded before)."""
    import torch
    from torch.utils import cpp_extension
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            "-fvisibility=hidden", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{p}" for p in inc), os.path.join(CSRC, "bind.cpp"), "-o", out, f"-L{lib}",
            "-lc10", "-ltorch_cpu", "-ltorch", "-ltorch_python"]


def _run(cmd: list[str]) -> tuple[int, str]:
    try:
        p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:   # a compiler that is not there fails its own command only
        return 127, str(e)
    out = "\n".join(l for l in p.stdout.splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    return p.returncode, out


def build(verbose: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()
    objs, cmds = [], []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        cmds.append([cc, *compile_flags(), "-c", os.path.join(CSRC, src), "-o", obj])
    binding = _bind_command()
    cmds += [binding] if binding else []
    jobs = jobs or min(len(cmds), max(1, (os.cpu_count() or 2) // 2))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        results = list(ex.map(_run, cmds))

    def check(cmd, rc, out):
        if verbose or rc:
            print(" ".join(cmd), file=sys.stderr)
            if out.strip():
                print(out, file=sys.stderr)
        if rc:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({rc}): {' '.join(cmd)}")

    for cmd, (rc, out) in zip(cmds[:len(objs)], results):
        check(cmd, rc, out)
    tmp = LIB + ".tmp"
    rc, out = _run([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp])
    if rc:
        print(out, file=sys.stderr)
        raise RuntimeError("link of libdora.so failed")
    os.replace(tmp, LIB)   # whatever becomes of the Python binding
    if binding:
        check(binding, *results[-1])
        os.replace(BIND + ".tmp", BIND)
    return LIB


def _bind_command() -> list[str] | None:
    try:
        return bind_command(BIND + ".tmp")
    except ImportError as e:
        print(f"_bind.so is not built: {e} (libdora.so does not need it)", file=sys.stderr)
        return None


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
