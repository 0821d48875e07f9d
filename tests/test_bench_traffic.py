"""Host test: bench.py reports a profile's HBM traffic only for the sources it was
measured on, the header with the GEMM's pipeline among them."""
import hashlib
import json
import os
import sys

import pytest

pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


def test_traffic_is_that_of_the_sources(tmp_path, monkeypatch):
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    (tmp_path / "profiles").mkdir()

    def write(name, text):
        (tmp_path / name).write_text(text)
        return hashlib.sha256(text.encode()).hexdigest()

    summary = {"source": "k.hip", "source_sha256": write("k.hip", "kernel"),
               "headers_sha256": {"core.hpp": write("core.hpp", "pipeline")}, "bytes_per_launch": 123}
    (tmp_path / "profiles" / "t.json").write_text(json.dumps(summary))
    assert bench.measured_traffic("t.json") == 123
    assert bench.measured_traffic("other.json") is None
    write("core.hpp", "another pipeline")
    assert bench.measured_traffic("t.json") is None
    write("core.hpp", "pipeline")
    write("k.hip", "another kernel")
    assert bench.measured_traffic("t.json") is None


def test_gemm_summaries_name_the_pipeline():
    """The GEMM's kernel is in two files; a summary of its traffic names both."""
    where = os.path.join(bench.ROOT, "profiles")
    names = [n for n in os.listdir(where) if n.startswith("traffic_gemm_") and n.endswith(".json")]
    assert names
    for name in names:
        with open(os.path.join(where, name)) as f:
            tr = json.load(f)
        assert tr["source"].endswith("csrc/gemm.hip"), name
        assert [os.path.basename(h) for h in tr["headers_sha256"]] == ["gemm_core.hpp"], name
