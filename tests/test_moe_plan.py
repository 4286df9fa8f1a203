"""CPU tests of how a call on a block of experts (include/cbk_moe.h) is cut up (``ex_plan``): every shape that is accepted has
launches of fewer than 2^32 threads and a workspace whose parts are large enough and apart; with a host-only program
(tests/sanitize/moe_plan.cpp), built with AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "fly_decode_amd", "csrc")

pytestmark = pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")

Case = namedtuple("Case", "rows cols out count b b_down tokens k backward")
Plan = namedtuple("Plan", "Tc tile max_tiles one split_down split_dt split_x dw_parts s_stride d_stride tiles token_of slot_of place_of xpack ypack "
                          "h g s d dw bytes")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    srcs = [os.path.join(SAN, "moe_plan.cpp"), os.path.join(SAN, "stubs.cpp"), os.path.join(CSRC, "cbk_moe_host.cpp"),
            os.path.join(CSRC, "cbk_api.cpp"), os.path.join(CSRC, "cbk_ec_host.cpp")]
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-pthread", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", SAN,
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, *srcs, "-o", exe], check=True)

    def run(cases):
        text = "".join(" ".join(str(int(v)) for v in c) + "\n" for c in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0, r.stderr[-4000:]
        got = [Plan(*(int(v) for v in line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(cases)
        return got

    return run


def up(n, m):
    return -(-n // m) * m


def everything():
    widths = [(1, 1, 1), (64, 70, 33), (683, 1001, 1001), (2048, 4096, 4096), (65536, 64, 64), (1 << 18, 8, 1 << 18), (1 << 19, 64, 64),
              (1 << 20, 8, 8), (1 << 20, 1 << 20, 1 << 20), (8, 1 << 20, 8), (8, 8, 1 << 20)]
    return [Case(*w, count, b, b_down, T, k, backward) for w in widths for count in (1, 8, 61, 128, 480, 1024)
            for b, b_down in ((0, 1), (13, 13), (13, 14), (14, 14), (16, 15)) for T in (1, 7, 45, 481, 700, 2048, 16384, 1 << 20, (1 << 31) - 1)
            for k in (1, 5, 64) for backward in (0, 1)]


def test_launches(plans):
    """What a product has of tiles, by the columns that each kernel's tile holds (of a pair half as many of the hidden)."""
    cases = everything()
    for c, p in zip(cases, plans(cases)):
        assert 1 <= p.Tc <= c.tokens and p.tile in (16, 64, 256), (c, p)
        slots = p.Tc * c.k
        assert slots <= max(65536, c.k) and p.max_tiles >= (c.k if p.one else min(c.count, slots) + slots // p.tile), (c, p)
        columns = 256 if p.tile == 256 else 128
        hidden = p.max_tiles * -(-up(c.rows, 64) // (columns // 2))
        if c.backward:
            others = [p.max_tiles * -(-c.rows // columns) * p.split_dt, p.max_tiles * -(-c.cols // columns) * p.split_x]
            assert p.dw_parts == -(-up(c.rows, 64) // (columns // 2)) * (2 if p.tile == 256 else 4)
        else:
            others = [p.max_tiles * -(-c.out // columns) * p.split_down]
        for units in (hidden, *others):
            assert (units + 7) // 8 * 8 * 512 < 1 << 32, (c, p)
        # k_experts_few: 16 hidden columns, its units numbered in 32 bits
        assert p.max_tiles * up(c.rows, 64) // 16 < 1 << 26, (c, p)


def test_workspace(plans):
    cases = everything()
    for c, p in zip(cases, plans(cases)):
        slots, F = p.Tc * c.k, up(c.rows, 64)
        need = {"tiles": 16 * p.max_tiles, "token_of": 4 * slots, "slot_of": 4 * slots, "place_of": 4 * slots, "xpack": p.Tc * up(c.cols, 64) * 2}
        if c.backward:
            assert p.s_stride >= slots * up(c.cols, 128) and p.d_stride >= slots * up(c.rows, 128)
            need.update(ypack=p.Tc * up(c.out, 64) * 2, d=p.split_dt * p.d_stride * 4, g=slots * 4 * F, s=p.split_x * p.s_stride * 4,
                        dw=slots * p.dw_parts * 4)
        else:
            assert p.s_stride >= slots * up(c.out, 128)
            need.update(h=slots * 2 * F, s=p.split_down * p.s_stride * 4)
        at = 4  # the number of tiles
        for name, size in sorted(need.items(), key=lambda n: getattr(p, n[0])):
            start = getattr(p, name)
            assert start >= at and start % 256 == 0, (c, p, name)
            at = start + size
        assert at <= p.bytes < 12 << 30, (c, p)


def test_wide_layers_take_chunks(plans):
    """Blocks of a million hidden columns with hundreds of experts in use: as many tokens at a time as a launch takes."""
    cases = [Case(1 << 20, 8, 8, 1024, b, 13, 2000, 1, 0) for b in (13, 14)] + [Case(1 << 20, 8, 8, 1024, 14, 14, 300, 1, 0)]
    first, second, small = plans(cases)
    assert first.Tc == second.Tc == 480 and first.tile == 16 and small.Tc == 300
