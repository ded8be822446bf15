"""The DRAM traffic of the bench's roofline: the committed captures are recognised by the sources of the
kernel that they were taken of, and by nothing else."""
import os
import shutil

import pytest

import bench
from conftest import ROOT

CAPTURES = [("b1", "expert_dec"), ("b8", "expert_dec"), ("b64", "expert_dec"), ("prefill", "expert_wide")]


@pytest.fixture
def copy_of_tree(tmp_path, monkeypatch):
    for part in ("profiles", os.path.join("routed_moe_decode_gb300", "csrc")):
        shutil.copytree(os.path.join(ROOT, part), tmp_path / part)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path


@pytest.mark.parametrize("config,kernel", CAPTURES)
def test_committed_captures_are_of_the_sources(config, kernel):
    assert bench.profiled_traffic(config, kernel) > 1e6


@pytest.mark.parametrize("config,kernel", CAPTURES)
def test_only_the_kernels_own_sources_count(copy_of_tree, config, kernel):
    csrc = copy_of_tree / "routed_moe_decode_gb300" / "csrc"
    headers = bench.kernel_headers(kernel)
    assert "moe_common.cuh" in headers and "moe_kernels.cuh" in headers
    with open(csrc / "another_operator.cuh", "w") as f:
        f.write("#pragma once\n")
    with open(csrc / "kv4_common.cuh", "a") as f:
        f.write("// changed\n")
    assert bench.profiled_traffic(config, kernel) is not None
    for name in [f"{kernel}.cu", *headers]:
        text = (csrc / name).read_text()
        (csrc / name).write_text(text + "// changed\n")
        assert bench.profiled_traffic(config, kernel) is None, name
        (csrc / name).write_text(text)
    assert bench.profiled_traffic(config, kernel) is not None
