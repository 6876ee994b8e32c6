"""The recorded counter figures that bench.py prints: valid for the sources and flags they were taken
on, whatever else the library is built from (CPU)."""
import json
import os

import pytest

import bench
from linear_attention_recurrence_05_amd import build as kbuild

RECORDS = json.load(open(os.path.join(bench.ROOT, "profiles", "traffic.json")))["records"]


@pytest.mark.parametrize("key", sorted(RECORDS))
def test_records_outlive_other_sources(key, monkeypatch):
    """Another source in the library, or another flag for it, leaves a record as it is; another flag for
    its own sources does not."""
    sources = RECORDS[key]["sources"]
    assert any(s.endswith(".hip") for s in sources) and not any(s.endswith("build.py") for s in sources)
    before = bench.source_fingerprint(sources)
    monkeypatch.setattr(kbuild, "SOURCES", kbuild.SOURCES + ["another.hip"])
    monkeypatch.setitem(kbuild.SOURCE_FLAGS, "another.hip", ["-O1"])
    assert bench.source_fingerprint(sources) == before
    own = os.path.basename(next(s for s in sources if s.endswith(".hip")))
    monkeypatch.setitem(kbuild.SOURCE_FLAGS, own, kbuild.SOURCE_FLAGS.get(own, []) + ["-O1"])
    assert bench.source_fingerprint(sources) != before


def test_a_record_of_other_sources_is_not_used(monkeypatch):
    key = sorted(RECORDS)[0]
    field = "bytes" if "bytes" in RECORDS[key] else "value"
    monkeypatch.setattr(bench, "source_fingerprint", lambda sources: RECORDS[key]["sha256_16"])
    assert bench.recorded(key, field) == RECORDS[key][field]
    monkeypatch.setattr(bench, "source_fingerprint", lambda sources: "0" * 16)
    assert bench.recorded(key, field) is None
    assert bench.recorded("no such record", "bytes") is None
