"""bench.py reports a kernel's DRAM traffic only for the sources that it was captured
from, and says so where they changed."""
import hashlib
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_current_and_stale_captures(tmp_path, monkeypatch, capsys):
    (tmp_path / "profiles").mkdir()
    (tmp_path / "a.cu").write_text("one")
    entry = dict(sources=["a.cu"], sha256=hashlib.sha256(b"one").hexdigest(), dram_bytes=300, algorithmic_bytes=200)
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps({"k@w": entry}))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_traffic("k", "w", 400) == 600
    assert bench.kernel_traffic("other", "w", 400) is None
    assert capsys.readouterr().err == ""
    (tmp_path / "a.cu").write_text("two")
    assert bench.kernel_traffic("k", "w", 400) is None
    out = capsys.readouterr()
    assert "k@w" in out.err and "changed" in out.err and out.out == ""
