"""Builds libmoestep.so (HIP kernels + C ABI) in-tree for gfx950 with hipcc, and _marshal.so (the
binding's compiled part, host code only) with g++."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libmoestep.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # keep the compiler from forming packed fp32 ALU ops (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.hip")))


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{msgs}")
    if msgs.strip() and verbose:
        print(msgs, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compiles every source (side by side) and links.  The library and _marshal.so share argument
    structs, so both are put in their places, whole, once everything has been built."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    compiled = [f for f in HIPCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="moestep_") as tmp, \
            concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objects = [os.path.join(tmp, os.path.basename(f) + ".o") for f in sources()]
        jobs = [pool.submit(_run, [hipcc, *compiled, "-I", os.path.join(ROOT, "include"), "-c", f, "-o", o], verbose)
                for f, o in zip(sources(), objects)]
        marshal = os.path.join(tmp, "_marshal.so")
        jobs.append(pool.submit(build_marshal, marshal, verbose))
        for j in jobs:
            j.result()
        _run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", *objects, "-o", LIB + ".tmp"], verbose)
        shutil.copy(marshal, MARSHAL + ".tmp")
    os.replace(LIB + ".tmp", LIB)
    os.replace(MARSHAL + ".tmp", MARSHAL)
    return LIB


def build_marshal(out: str, verbose: bool = False) -> None:
    import torch

    at = os.path.dirname(torch.__file__)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(at, "include"),
           "-isystem", os.path.join(at, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(PKG, "csrc", "marshal.cpp"), "-o", out,
           "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    _run(cmd, verbose)


if __name__ == "__main__":
    print(build(verbose=True))
