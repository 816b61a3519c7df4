"""The kernels' inline assembly, read as text: registers that the compiler owns
and that a clobber list cannot name are given back."""
import glob
import os
import re

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "sparse_bf16_delta_amd", "csrc", "*")))


def asm_statements():
    for path in SOURCES:
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", text, flags=re.S):
            code = "".join(re.findall(r'"([^"]*)"', m.group(1).split(":")[0]))
            yield os.path.basename(path), [line.strip() for line in
                                           code.replace("\\t", "").split("\\n")]


def test_m0_is_given_back():
    found = 0
    for name, lines in asm_statements():
        if not any(re.match(r"s_mov_b32 m0,", line) for line in lines):
            continue
        found += 1
        saved = re.fullmatch(r"s_mov_b32 (%\d+), m0", lines[0])
        assert saved, (name, lines)
        assert lines[-1] == f"s_mov_b32 m0, {saved.group(1)}", (name, lines)
    assert found == 1
