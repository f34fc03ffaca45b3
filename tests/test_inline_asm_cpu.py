"""Inline assembly of the kernels (CPU: the sources are read)."""
from __future__ import annotations

import os
import re

from mxfp4_routed_expert_route_amd import build as build_mod


def _asm_statements():
    for name in sorted(os.listdir(build_mod.CSRC)):
        if name.endswith((".hip", ".h")):
            text = open(os.path.join(build_mod.CSRC, name)).read()
            for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\((.*?)\);", text, flags=re.S):
                yield name, m.group(1)


def test_m0_is_an_operand_and_never_written():
    # m0 is the compiler's register and cannot be named as clobbered: a statement that needs a
    # value in it takes it as an operand, and the compiler knows what m0 then holds
    seen = 0
    for name, text in _asm_statements():
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split('"memory"')[0].split('::')[0]))
        code = code.replace("\\n", "\n").replace("\\t", " ")
        for line in code.split("\n"):
            words = line.replace(",", " ").split()
            assert words[1:2] != ["m0"], (name, line)
            if "lds" in words:      # a load that writes LDS, at m0
                seen += 1
                assert '"{m0}"(' in text, (name, line)
    assert seen >= 3
