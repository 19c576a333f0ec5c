"""The library and the binding's compiled part belong together: they are put in place together, and
a pair that was built from different headers is refused."""
import ctypes as C
import os

import pytest

import asynchronous_moe_expert_amd as M
from asynchronous_moe_expert_amd import _native as N
from asynchronous_moe_expert_amd import build as B

SIZE_FN, VERSION_FN = C.CFUNCTYPE(C.c_size_t, C.c_int), C.CFUNCTYPE(C.c_int)


@pytest.fixture(scope="module")
def lib():
    if not (os.path.exists(M.LIB_PATH) and os.path.exists(B.MARSHAL)):
        B.build()
    return M.load()


def address(f):
    return C.cast(f, C.c_void_p).value


def test_marshal_refuses_a_library_of_another_header(lib):
    from asynchronous_moe_expert_amd import _marshal as m

    entries = [address(getattr(lib, name)) for name in N._HOME]
    strerror, version, size = (address(getattr(lib, name)) for name in ("moe_strerror", "moe_version", "moe_struct_size"))
    for which in range(5, 12):
        other = SIZE_FN(lambda i, which=which: lib.moe_struct_size(i) + 8 * (i == which))
        with pytest.raises(M.MoeError, match=rf"layout mismatch \(id {which}\)"):
            m.setup(M.MoeError, strerror, version, address(other), *entries)
    newer = VERSION_FN(lambda: lib.moe_version() + 1)
    with pytest.raises(M.MoeError, match="version"):
        m.setup(M.MoeError, strerror, address(newer), size, *entries)
    m.setup(M.MoeError, strerror, version, size, *entries)  # the real pair agrees


def script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(0o755)
    return str(path)


@pytest.mark.parametrize("fails", ["hipcc -c", "hipcc link", "g++", "nothing"])
def test_build_replaces_both_files_or_neither(tmp_path, monkeypatch, fails):
    """Stand-ins for the compilers that write `new` to their output, or fail at one step."""
    write = 'while [ $# -gt 0 ]; do [ "$1" = -o ] && echo new > "$2"; shift; done\n'
    steps = {"hipcc -c": 'case "$*" in *" -c "*) exit 1;; esac\n', "hipcc link": 'case "$*" in *" -c "*) ;; *) exit 1;; esac\n'}
    monkeypatch.setenv("HIPCC", script(tmp_path / "hipcc", steps.get(fails, "") + write))
    monkeypatch.setenv("CXX", script(tmp_path / "gxx", ("exit 1\n" if fails == "g++" else "") + write))
    lib, marshal = tmp_path / "libmoestep.so", tmp_path / "_marshal.so"
    monkeypatch.setattr(B, "LIB", str(lib))
    monkeypatch.setattr(B, "MARSHAL", str(marshal))
    for f in (lib, marshal):
        f.write_text("old\n")
    if fails == "nothing":
        B.build()
    else:
        with pytest.raises(RuntimeError, match="failed"):
            B.build()
    want = "new\n" if fails == "nothing" else "old\n"
    assert lib.read_text() == marshal.read_text() == want
