"""Wait states behind matrix instructions in the linear-attention kernels.

A matrix instruction's result must not be read by another kind of instruction
before it has landed, and it is the compiler that has to put the wait states
there.  It has left them out where a branch led from the product to its reader
past inline assembly: the reader then took one register too early.  So the
assembly that the sources compile to is checked, along every path.
"""
import os
import re
import subprocess

import pytest

from gated_deltanet_recurrence_delta_amd import build as hip_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# instructions, s_nop's count among them, between product and reader
WAIT = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}


def _registers(text):
    found = set()
    for a, b in re.findall(r"\bv\[(\d+):(\d+)\]", text):
        found |= set(range(int(a), int(b) + 1))
    return found | {int(a) for a in re.findall(r"\bv(\d+)\b", text)}


def _functions(text):
    """(name, instructions, label -> index) of each function."""
    for m in re.finditer(r"^(\w+):\s*; @\1$", text, re.M):
        code, labels = [], {}
        for line in text[m.start():text.index(".Lfunc_end", m.start())].split("\n"):
            line = line.split(";")[0].strip()
            if re.match(r"\.LBB\w+:", line):
                labels[line[:-1]] = len(code)
            elif line and not line.startswith(".") and not line.endswith(":"):
                code.append(line)
        yield m.group(1), code, labels


def early_readers(text):
    bad, products = [], 0
    for name, code, labels in _functions(text):
        for n, line in enumerate(code):
            op = line.split()[0]
            if not op.startswith("v_mfma"):
                continue
            products += 1
            todo, seen = [(n + 1, 0, frozenset(_registers(line.split(None, 1)[1].split(",")[0])))], set()
            while todo:
                k, waited, live = todo.pop()
                if k >= len(code) or waited >= WAIT[op] or not live or (k, waited, live) in seen:
                    continue
                seen.add((k, waited, live))
                x, _, args = code[k].partition(" ")
                if x == "s_nop":
                    todo.append((k + 1, waited + int(args, 0) + 1, live))
                    continue
                if x in ("s_branch", "s_endpgm"):
                    if x == "s_branch":
                        todo.append((labels[args.strip()], waited + 1, live))
                    continue
                if x.startswith("s_cbranch"):
                    todo.append((labels[args.strip()], waited + 1, live))
                elif x.startswith(("v_", "ds_", "buffer_", "global_", "flat_")):
                    first, _, rest = args.partition(",")
                    writes = not x.startswith(("ds_write", "buffer_store", "global_store")) and not args.endswith("lds")
                    if not x.startswith("v_mfma") and _registers(rest if writes else args) & live:
                        bad.append((name, line, waited, code[k]))
                        continue
                    if writes:
                        live = live - _registers(first)
                todo.append((k + 1, waited + 1, live))
    return bad, products


def test_an_early_reader_is_seen():
    """Behind a branch, and no other."""
    text = """
f:                                      ; @f
	v_mfma_f32_16x16x4_f32 v[0:3], v8, v9, v[0:3]
	s_cbranch_scc1 .LBB0_2
	s_nop 7
	v_add_f32_e32 v5, v6, v7
.LBB0_2:
	ds_read_b32 v5, v6
	v_mul_f32_e32 v3, v4, v3
	s_endpgm
.Lfunc_end0:
"""
    bad, products = early_readers(text)
    assert products == 1 and [(b[2], b[3].split()[0]) for b in bad] == [(2, "v_mul_f32_e32")]
    assert early_readers(text.replace("ds_read_b32 v5, v6", "s_nop 8"))[0] == []


@pytest.mark.skipif(not os.path.exists(hip_build.HIPCC), reason="no hipcc in this image")
def test_no_product_is_read_early(tmp_path):
    out = str(tmp_path / "linear.s")
    flags = [f for f in hip_build.FLAGS if f not in ("-shared",)]
    src = os.path.join(hip_build.HERE, "csrc", "gdn_linear.hip")
    subprocess.run([hip_build.HIPCC, *flags, "-S", "--offload-device-only", src, "-o", out], check=True,
                   stderr=subprocess.DEVNULL)
    bad, products = early_readers(open(out).read())
    assert products > 1000
    assert not bad, bad[:5]
