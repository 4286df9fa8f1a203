"""CPU tests of the committed traffic records: each was taken on the kernels as they are, so the benchmark
line cites it."""
import glob
import json
import os
import shutil

import pytest

from fly_decode_amd import profiling

RECORDS = sorted(glob.glob(os.path.join(profiling.PROFILES, "traffic_*.json")))


def test_there_are_records():
    assert len(RECORDS) >= 18


@pytest.mark.parametrize("path", RECORDS, ids=os.path.basename)
def test_a_record_is_of_the_current_kernels(path):
    with open(path) as f:
        rec = json.load(f)
    assert rec["source_sha256"] == profiling.kernel_source_sha256(rec["kernel"])


@pytest.mark.parametrize("kernel,files", [
    ("k_gemv_rows", {"cbk_kernels.hip", "cbk_device.h"}), ("k_decode_fast", {"cbk_kernels.hip", "cbk_device.h"}),
    ("k_enc_pack", {"cbk_encode.hip"}), ("k_ec_decode", {"cbk_ec.hip"}),
    ("k_mm", {"cbk_nn.hip", "cbk_nn_device.h", "cbk_device.h"}),
    ("k_fused", {"cbk_nn_fused.h", "cbk_nn_device.h", "cbk_device.h"})])
def test_a_change_to_what_a_kernel_is_built_from_makes_its_records_stale(tmp_path, monkeypatch, kernel, files):
    """Its own source and the device helpers that it includes, and no other file."""
    here, csrc = profiling.CSRC, str(tmp_path / "csrc")
    shutil.copytree(here, csrc)
    for name in ("CSRC", "ENCODER_SOURCE", "EC_SOURCE"):
        monkeypatch.setattr(profiling, name, getattr(profiling, name).replace(here, csrc))
    before = profiling.kernel_source_sha256(kernel)
    seen = set()
    for name in os.listdir(csrc):
        path = os.path.join(csrc, name)
        with open(path) as f:
            text = f.read()
        with open(path, "a") as f:
            f.write("// changed\n")
        if profiling.kernel_source_sha256(kernel) != before:
            seen.add(name)
        with open(path, "w") as f:
            f.write(text)
    assert seen == files
