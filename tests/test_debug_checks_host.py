"""The debug build's promise on the host: in the kernels of the serving calls no buffer of global
memory is subscripted but behind the bounds check.  (That the checked kernels give the same results
and report nothing is tested on the GPU.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_81_b200", "csrc")
FILES = ["fa_pages_sm100.cuh", "fa_rope_sm100.cuh", "fa_varlen_sm100.cuh"]


def code_of(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", src)


def members(code):
    """The pointer members of the parameter structs: what a kernel is given of global memory."""
    names = set()
    for body in re.findall(r"struct (?:PageTables|\w*Params) \{(.*?)\n\};", code, re.S):
        for line in body.split(";"):
            if "(" not in line and "*" in line:
                names |= set(re.findall(r"\*\s*(\w+)", line))
    return names


@pytest.mark.parametrize("name", FILES)
def test_no_buffer_is_subscripted_past_the_check(name):
    code = code_of(name)
    names = members("".join(code_of(f) for f in FILES))
    assert {"block_table", "copies", "free_ids", "plan", "positions", "q_out"} <= names
    raw = [line.strip() for line in code.split("\n")
           if re.search(rf"\b[pm](?:\.\w+)?\.(?:{'|'.join(sorted(names))})\[(?!\d+\])", line) and "in_bounds(" not in line]
    assert raw == [], raw


def test_the_accessors_check():
    code = code_of("fa_common.cuh")
    for f in ("read_at", "write_at"):
        body = re.search(rf"{f}\(.*?\n\}}", code, re.S).group(0)
        assert "in_bounds(i, n)" in body
