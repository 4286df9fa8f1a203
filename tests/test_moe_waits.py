"""The compiled order of the experts' products (``cbk_moe_mm.hip``).

An interval of their loop ends with a wait that may leave the words of a later slice in flight, or, where none are asked
for, nothing.  Either way every copy into LDS has to have landed: in the device assembly, at every barrier behind
multiplications, no more vector loads may be allowed in flight than stand behind the last copy.

The waves of ``k_experts_few`` wait for their own copies by counting what they asked for later: the loads of a step's tokens
and the copies of two items, none of which the compiler may have dropped or moved."""
import os
import re
import shutil
import subprocess

import pytest

from fly_decode_amd import build


def barriers(text):
    """(kernel, vector memory operations since the last barrier, allowed in flight) at every barrier of a block that
    multiplies and copies."""
    for name in re.findall(r"^(_ZN3cbk\S*k_experts(?:_many)?I\S*):", text, re.M):
        body = text[text.index("\n" + name + ":"):]
        body = body[:body.index(".Lfunc_end")]
        for block in re.split(r"\n(?=\.LBB)", body):
            if "v_mfma" not in block:
                continue
            ops, allowed = "", None
            for line in block.split("\n"):
                words = line.split(";")[0].split()
                if not words:
                    continue
                if words[0].startswith(("buffer_load", "global_load", "buffer_store", "global_store")):
                    ops += "C" if "lds" in words else "L"
                    allowed = None
                elif words[0] == "s_waitcnt" and "vmcnt" in line:
                    allowed = int(re.search(r"vmcnt\((\d+)\)", line).group(1))
                elif words[0] == "s_barrier":
                    if "C" in ops:
                        yield name, ops, allowed
                    ops, allowed = "", None


def covered(ops, allowed):
    return allowed is not None and allowed <= len(ops) - 1 - ops.rindex("C")


def check_counted(name, text):
    """The loop's two waits for 12 operations: in front of the first a step's tokens and an item's copies, between them
    another item's copies.  (What else is asked for in between only makes a wait a stricter one.)"""
    body = text[text.index("\n" + name + ":"):]
    ops = ""
    for line in body[:body.index(".Lfunc_end")].split("\n"):
        words = line.split(";")[0].split()
        if not words:
            continue
        if words[0].startswith(("buffer_load", "global_load")):
            ops += "C" if "lds" in words else "L" if words[0].endswith("dwordx4") else "l"
        elif words[0] == "s_waitcnt" and "vmcnt(12)" in line:
            ops += "W"
    before, between, _ = ops.split("W")
    assert before.endswith("LLLLCCCC") and between.count("C") == 4 and "L" not in between, (name, ops)


def test_rule():
    assert covered("CLLLL", 4) and covered("CCLL", 0) and covered("C", 0)
    assert not covered("CCC", 4) and not covered("CLLLL", None) and not covered("LLLLC", 4)


@pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="needs hipcc")
def test_copies_are_waited_for(tmp_path):
    out = str(tmp_path / "mm.s")
    subprocess.run([build.HIPCC, *build.DEVICE_FLAGS, *build.COMMON, "-S", "--offload-device-only", "-o", out,
                    os.path.join(build.CSRC, "cbk_moe_mm.hip")], check=True, capture_output=True)
    with open(out) as f:
        text = f.read()
    kernels = set()
    for name, ops, allowed in barriers(text):
        kernels.add(name)
        assert covered(ops, allowed), (name, ops, allowed)
    # (those that read their tables through the caches branch at it, and always wait for everything)
    every = {n for n in re.findall(r"^(_ZN3cbk\S*k_experts(?:_many)?I\S*):", text, re.M)
             if "_many" in n or not n.split("Ev")[0].endswith("ELb1EE")}
    assert kernels == every and len(every) == 10
    few = re.findall(r"^(_ZN3cbk\S*k_experts_fewI\S*):", text, re.M)
    assert len(few) == 5
    for name in few:
        check_counted(name, text)
