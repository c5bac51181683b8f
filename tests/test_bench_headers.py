"""The sources that bench.py's hash leaves out are those that no workload's kernel
includes, by their own name or through another header, and a change to any of them
keeps the hash."""
import os
import re
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

CSRC = os.path.join(ROOT, "segmented_gather_lora_amd", "csrc")


def included(name):
    with open(os.path.join(CSRC, name)) as f:
        return set(re.findall(r'^\s*#\s*include\s+"([^"]+)"', f.read(), re.M))


def test_measured_sources_include_measured_headers_alone():
    files = sorted(os.listdir(CSRC))
    measured = [f for f in files if f not in bench.NOT_MEASURED]
    assert set(bench.NOT_MEASURED) <= set(files) and measured
    for f in measured:
        assert not included(f) & set(bench.NOT_MEASURED), f
    # (and those that are left out do meet each other: the pattern finds includes)
    assert "lora_mx.h" in included("lora_linear.h") and "lora_gemm.h" in included("lora_mx.h")


@pytest.mark.parametrize("name", sorted(bench.NOT_MEASURED))
def test_hash_stays_when_others_change(name, tmp_path, monkeypatch):
    to = os.path.join(str(tmp_path), "segmented_gather_lora_amd", "csrc")
    shutil.copytree(CSRC, to)
    before = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    with open(os.path.join(to, name), "a") as f:
        f.write("\n// changed\n")
    assert bench.kernel_source_hash() == before
