"""Inline assembly in the kernels: what a statement writes beside its outputs is named in its list."""
import glob
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "asynchronous_moe_expert_amd", "csrc")


def statements():
    for f in sorted(glob.glob(os.path.join(SRC, "*.h*"))):
        for m in re.finditer(r"asm volatile\((.*?)\);", open(f).read(), re.S):
            yield os.path.basename(f), m.group(1)


def test_registers_that_are_written_are_named():
    found = 0
    for where, text in statements():
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text))
        if re.search(r"\bm0\s*,", code):
            found += 1
            assert '"m0"' in text, (where, text)
        if re.search(r"\bs_(add|sub|addc|subb|and|or|lshl)_[ub]\d+", code):
            assert '"scc"' in text, (where, text)
    assert found  # the copies into LDS
