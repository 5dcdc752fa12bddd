"""bench.py's measured HBM traffic: reported for the sources and flags it was measured with, and only for those."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("key", sorted(bench.MEASURED_TRAFFIC))
def test_traffic_of_the_present_sources(key):
    assert bench.measured_traffic(key) == bench.MEASURED_TRAFFIC[key]
    with open(os.path.join(ROOT, bench.MEASURED_TRAFFIC[key]["profile"])) as f:
        text = f.read()
    for what in ("sha16", "flags_sha16"):
        assert bench.MEASURED_TRAFFIC[key][what] in text
    assert f"{bench.MEASURED_TRAFFIC[key]['bytes_per_launch']:,}" in text


def test_only_flags_of_the_build_script_count(tmp_path, monkeypatch):
    """Another build script with the same flags leaves the entries valid; other flags, or another source, do not."""
    script = tmp_path / "build.py"
    shutil.copy(bench.BUILD_SCRIPT, script)
    script.write_text(script.read_text() + "\n# one more host source\n")
    flags = bench.flags_sha()
    assert bench.flags_sha(str(script)) == flags
    script.write_text(script.read_text() + "\nDEVICE_FLAGS = DEVICE_FLAGS[:-2]\n")
    assert bench.flags_sha(str(script)) != flags
    monkeypatch.setattr(bench, "flags_sha", lambda: "0" * 16)
    assert bench.measured_traffic("rabit") is None
    monkeypatch.undo()
    monkeypatch.setattr(bench, "source_sha", lambda name: "0" * 16)
    assert bench.measured_traffic("rabit") is None
