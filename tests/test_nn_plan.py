"""CPU tests of how a call of the operators in include/cbk_nn.h is cut up (``nn_plan``): which way of
computing a shape takes, checked with a host-only program (tests/sanitize/plan.cpp)."""
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "fly_decode_amd", "csrc")

pytestmark = pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")

LINEAR, BLOCK, HEAD = 0, 1, 2
Plan = namedtuple("Plan", "fused grid pieces rows in_order bytes")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    srcs = [os.path.join(SAN, "plan.cpp"), os.path.join(SAN, "stubs.cpp"), os.path.join(CSRC, "cbk_nn_host.cpp"),
            os.path.join(CSRC, "cbk_api.cpp"), os.path.join(CSRC, "cbk_ec_host.cpp")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", SAN,
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, *srcs, "-o", exe], check=True)

    def run(cases):
        """cases: (op, rows, cols, b, b of a pair's second tensor, tokens); a Plan for each."""
        text = "".join(" ".join(str(v) for v in c) + "\n" for c in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        got = [Plan(*(int(v) for v in line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(cases)
        return got

    return run


def test_every_piece_is_decoded_in_the_streams_order(plans):
    """Widths 1 to 15: no shape's pieces fall to the generic kernel, which is for other widths."""
    shapes = [(rows, cols) for rows in (1, 1000, 4096, 11008, 16384, 32000, 32768, 65536, 128256, 131072, 1 << 20)
              for cols in (1, 63, 64, 1001, 4096, 4097, 5120, 8192, 11008, 16384, 28672, 65536, 1 << 19, (1 << 19) + 1, 1 << 20)
              if rows * cols <= 1 << 35]  # index words of 64 GB are more than its chunk numbers hold
    cases = [(op, rows, cols, b, b2, tokens) for rows, cols in shapes for op in (LINEAR, BLOCK, HEAD)
             for b, b2 in ((1, 15), (13, 13)) for tokens in (385, 2048)]
    for case, p in zip(cases, plans(cases)):
        assert p.fused == 0 and p.in_order == 1, (case, p)


def test_up_to_384_tokens_are_decoded_on_the_way(plans):
    """Widths 8 to 14: every number of tokens up to the limit that the row length and the pair's widths give."""
    cases = [(op, 4096, cols, b, b2, tokens)
             for b in range(8, 15) for op, b2 in ((LINEAR, b), (HEAD, b), (BLOCK, b), (BLOCK, 8 if b > 8 else 9))
             for cols, most in ((4096, 384), (1023, 128 if op == BLOCK and b != b2 else 256))
             for tokens in range(1, most + 1)]
    for case, p in zip(cases, plans(cases)):
        assert p.fused >= case[5] and p.grid >= 256, (case, p)
