"""The benchmark's recorded HBM traffic (host logic, no GPU): reported while the sources it was taken on are the same, and
those are the files of the kernels it is about, so that work beside them does not take the figure away."""

import hashlib
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = "bit_quantized_finetuning_amd/csrc/"
OWN = {bench.FWD_TRAFFIC_RECORD: {"gemm.hip", "lora_wide.hip", "api.cpp", "common.h", "tiles.h"},
       bench.TRAFFIC_RECORD: {"gemv.hip", "gemv_body.inc", "common.h"}}


@pytest.mark.parametrize("record", list(OWN))
def test_records_are_about_their_kernels_sources(record):
    with open(record) as f:
        rec = json.load(f)
    assert {s.removeprefix(CSRC) for s in rec["sources"]} == OWN[record]
    for prefix in ("", "grouped_"):
        if prefix and prefix + "launches" not in rec:
            continue
        assert rec[prefix + "traffic_bytes_per_launch"] > 0 and rec[prefix + "launches"] > 0
    raw = rec["fetch_scale"] * rec["fetch_kib_per_launch_raw"] + rec["write_scale"] * rec["write_kib_per_launch_raw"]
    assert abs(rec["traffic_bytes_per_launch"] / (raw * 1024) - 1) < 1e-4


def test_a_record_is_reported_while_its_sources_are_the_same(tmp_path):
    src = os.path.relpath(tmp_path / "kernel.hip", ROOT)
    (tmp_path / "kernel.hip").write_text("one")
    rec = tmp_path / "record.json"
    rec.write_text(json.dumps({"sources": [src], "sources_sha256": hashlib.sha256(b"one").hexdigest(), "traffic_bytes_per_launch": 7}))
    assert bench.recorded_traffic(str(rec)) == 7
    (tmp_path / "kernel.hip").write_text("two")
    assert bench.recorded_traffic(str(rec)) is None
