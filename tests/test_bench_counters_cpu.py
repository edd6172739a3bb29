"""The benchmark takes the GEMM's HBM traffic from committed counters only while
the code they were taken on is the current one (no GPU)."""
import json
import os
import re

import pytest

pytest.importorskip("torch")

import bench  # noqa: E402


def device_headers(path, seen):
    """`path` and the headers of its folder that it includes and that hold device
    code."""
    text = open(path, encoding="utf-8").read()
    if path in seen or "__device__" not in text:
        return seen
    seen.add(path)
    for name in re.findall(r'#include "([^"/]+)"', text):
        device_headers(os.path.join(os.path.dirname(path), name), seen)
    return seen


def test_hash_covers_what_the_gemm_is_built_from():
    gemm = next(p for p in bench.GEMM_SOURCES if p.endswith("gemm.hip"))
    assert device_headers(gemm, set()) == set(bench.GEMM_SOURCES)


def test_traffic_only_from_the_current_code(tmp_path, monkeypatch):
    source = tmp_path / "gemm.hip"
    source.write_text("int x; // one\n")
    counters = tmp_path / "counters.json"
    monkeypatch.setattr(bench, "GEMM_SOURCES", [str(source)])
    monkeypatch.setattr(bench, "COUNTERS_FILE", str(counters))
    assert bench.traffic_from_counters() is None
    counters.write_text(json.dumps({"gemm_code_sha256": bench.code_hash([str(source)]),
                                    "hbm_bytes_per_launch": 5}))
    assert bench.traffic_from_counters() == 5
    source.write_text("/* another comment */ int  x;\n")
    assert bench.traffic_from_counters() == 5
    source.write_text("int y;\n")
    assert bench.traffic_from_counters() is None
