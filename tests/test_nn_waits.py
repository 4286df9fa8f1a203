"""The compiled order of the product that decodes on the way (``cbk_nn_fused.h``).

Its main loop ends each interval with a wait that lets the last NL vector loads, the words of a
later slice, stay in flight.  That covers the copies into LDS only if they stand before those loads
in the compiled code, so the device assembly of every instantiation is checked for it.
"""
import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

from fly_decode_amd import build

CSRC = os.path.join(os.path.dirname(os.path.abspath(build.__file__)), "csrc")
WIDTHS = range(8, 15)


def _assembly(width, folder):
    out = os.path.join(folder, f"{width}.s")
    subprocess.run([build.HIPCC, *build.DEVICE_FLAGS, *build.COMMON, "-S", "--offload-device-only", "-o", out,
                    os.path.join(CSRC, f"cbk_nn_fused_{width}.hip")], check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def intervals(text):
    """(kernel, vector memory operations since the last barrier, allowed in flight, whether the wait
    stands behind all of them) at every barrier of a loop that multiplies."""
    for name in re.findall(r"^(_ZN3cbk\S*k_fusedI\S*):", text, re.M):
        body = text[text.index("\n" + name + ":"):]
        body = body[:body.index(".Lfunc_end")]
        for block in re.split(r"\n(?=\.LBB)", body):
            label = block.split(":")[0].strip()
            if "v_mfma" not in block or not re.search(r"s_cbranch\S* " + re.escape(label) + r"\b", block):
                continue
            ops, allowed, last = "", None, False
            for line in block.split("\n"):
                words = line.split(";")[0].split()
                if not words:
                    continue
                if words[0].startswith(("buffer_load", "global_load", "buffer_store", "global_store")):
                    ops += "C" if "lds" in words else "L"
                    last = False
                elif words[0] == "s_waitcnt" and "vmcnt" in line:
                    allowed, last = int(re.search(r"vmcnt\((\d+)\)", line).group(1)), True
                elif words[0] == "s_barrier":
                    yield name, ops, allowed, last
                    ops, allowed, last = "", None, False


def covered(ops, allowed, last):
    return "C" in ops and last and allowed <= len(ops) - 1 - ops.rindex("C")


def test_rule():
    assert covered("CLL", 2, True) and covered("CCL", 1, True) and covered("CLL", 0, True)
    assert not covered("LLC", 2, True) and not covered("CLLC", 2, True)
    assert not covered("CLL", 2, False) and not covered("LL", 2, True)


@pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="needs hipcc")
def test_copies_are_waited_for(tmp_path):
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        texts = list(pool.map(lambda b: _assembly(b, str(tmp_path)), WIDTHS))
    kernels = set()
    for text in texts:
        for name, ops, allowed, last in intervals(text):
            kernels.add(name)
            assert covered(ops, allowed, last), (name, ops, allowed, last)
    assert len(kernels) == len(WIDTHS) * 7 * 4  # token tiles; orientation and ragged rows
