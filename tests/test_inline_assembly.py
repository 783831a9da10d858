"""CPU test of the kernels' sources: inline assembly holds waits for loads and orders memory accesses,
nothing else (an empty statement may hold a value in a register: the instructions around it are the
compiler's). The compiler counts the cycles that a matrix instruction's result takes, and those of every
other instruction, for its own instructions only; assembly that reads or writes a vector register would need
waits of its own, counted by hand, and a load written so could land in a register that is in use again."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "activation_sparse_decode_rank_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path, encoding="utf-8").read()
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\((.*?)\);", text, re.S):
            yield os.path.basename(path), m[1]


def test_inline_assembly_with_instructions_touches_no_vector_register():
    seen = list(statements())
    assert len(seen) > 5
    for name, what in seen:
        code = re.match(r'\s*((?:"[^"]*"\s*)+)', what)[1]
        words = re.sub(r'["\s]+', " ", code.replace("\\n", " ").replace("\\t", " ")).strip()
        assert words == "" or re.fullmatch(r"s_waitcnt [\w() %,&]*", words), (name, what)
        assert words == "" or not re.search(r'"[+=&]*[va]"', what), (name, what)
