"""The hash that ties bench.py's counted traffic to the kernels covers the sources
of the kernels that its workloads launch, and no others."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("name,counts", [("lora_shrink.hip", True), ("lora_expand.hip", True), ("lora_internal.h", True),
                                         ("lora_linear.hip", False), ("lora_loss.hip", False), ("lora_gemm.h", False)])
def test_hash_follows_the_workloads_kernels(name, counts, tmp_path, monkeypatch):
    to = os.path.join(str(tmp_path), "segmented_gather_lora_amd", "csrc")
    shutil.copytree(os.path.join(ROOT, "segmented_gather_lora_amd", "csrc"), to)
    before = bench.kernel_source_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash() == before
    with open(os.path.join(to, name), "a") as f:
        f.write("\n// changed\n")
    assert (bench.kernel_source_hash() != before) == counts


def test_operators_sources_reach_no_workload():
    """None of the workloads' kernels includes what the hash leaves out."""
    csrc = os.path.join(ROOT, "segmented_gather_lora_amd", "csrc")
    for f in sorted(os.listdir(csrc)):
        if f not in bench.NOT_MEASURED:
            with open(os.path.join(csrc, f)) as fh:
                assert "lora_gemm.h" not in fh.read(), f
