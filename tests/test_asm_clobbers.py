"""Inline assembly names the fixed registers that it writes, so that the
compiler keeps nothing of its own in them."""
import glob
import os
import re

import pytest

from gated_deltanet_recurrence_delta_amd import build as hip_build

FIXED = ("m0", "vcc", "exec")


def unnamed(text):
    """(assembly, register) of each written fixed register that is no clobber."""
    bad = []
    for asm in re.findall(r"\basm\s+volatile\s*\((.*?)\)\s*;", text, re.S):
        parts = re.sub(r'"\s*"', "", asm)  # adjacent literals are one
        code = re.match(r'\s*"(.*?)"', parts, re.S)
        clobbers = parts.count(":") >= 3 and parts.rsplit(":", 1)[1] or ""
        for line in re.split(r"\\n|\\t", code.group(1) if code else ""):
            words = line.replace(",", " ").split()
            for r in FIXED:
                if len(words) > 1 and words[1].split("_")[0] == r and f'"{r}"' not in clobbers:
                    bad.append((line, r))
    return bad


def test_an_unnamed_register_is_seen():
    head = 'asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 4" : : "s"(at)'
    assert unnamed(head + ");") == [("s_mov_b32 m0, %0", "m0")]
    assert unnamed(head + ' : "m0");') == [] and unnamed('asm volatile("s_nop 0");') == []


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(hip_build.HERE, "csrc", "*"))), ids=os.path.basename)
def test_fixed_registers_are_named(path):
    assert unnamed(open(path).read()) == []
