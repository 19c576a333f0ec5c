"""The SwiGLU kernels and the rule that gives rows their threads (cut from csrc/swiglu.hip), built for the host: for
every row length that the entry points take, each chunk of eight columns has one owner, and the gradient computed in
place equals the one that is not."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(HERE)
SRC = os.path.join(REPO, "asynchronous_moe_expert_amd", "csrc", "swiglu.hip")


def _source() -> str:
    src = open(SRC).read()
    at = src.index

    def cut(first, end):
        return src[at(first):at(end)]

    return "namespace moe {\n" + "\n".join([
        cut("// s = 1 / (1 + exp(-g))", "// One scale for a whole row"),
        cut("template <int DT, int S>\n__global__", "struct QuantizeJob {"),
        cut("// threads to a row and rows to a workgroup", "template <int XT, int OT>\nstatic int swiglu_by_kind"),
    ]) + "}  // namespace moe\n"


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("swiglu_host")
    open(d / "swiglu_kernels.inc", "w").write(_source())
    out = d / "swiglu_host"
    r = subprocess.run([gxx, "-std=c++20", "-O2", "-ffp-contract=off", "-D__HIP_PLATFORM_AMD__", f"-I{d}",
                        f"-I{os.path.join(HERE, 'host_build')}", f"-I{os.path.join(REPO, 'include')}",
                        "-I/opt/rocm/include", os.path.join(HERE, "host_build", "swiglu_host.cpp"), "-o", str(out),
                        "-lpthread"], capture_output=True, text=True)
    if r.returncode != 0:  # (a compiler that cannot build the kernels is a failure, not a skip)
        pytest.fail("host build failed: " + r.stderr[-1200:])
    return str(out)


def test_every_chunk_of_a_row_has_one_owner(exe):
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:]
