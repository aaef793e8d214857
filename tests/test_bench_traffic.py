"""The committed HBM traffic belongs to the sources as they are, and only what a kernel is built from can void it."""
import os
import shutil

import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.TRAFFIC_SOURCES))
def test_committed_traffic_applies(kernel):
    """A change to these kernels' sources takes new counters (bench.py --pmc-workload) along."""
    assert bench.traffic_from_summary(kernel) is not None


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "bit_matmul_amd" / "csrc"
    shutil.copytree(os.path.join(bench.ROOT, "bit_matmul_amd", "csrc"), csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return csrc


def test_a_header_that_a_kernel_does_not_include_voids_nothing(tree):
    before = {k: bench.kernel_sources_hash(k) for k in bench.TRAFFIC_SOURCES}
    (tree / "lq_another.h").write_text("#pragma once\n")
    (tree / "lq_rows.h").write_text((tree / "lq_rows.h").read_text() + "// more\n")
    assert {k: bench.kernel_sources_hash(k) for k in bench.TRAFFIC_SOURCES} == before


@pytest.mark.parametrize("header,kernels", [("lq_internal.h", set(bench.TRAFFIC_SOURCES)),
                                            ("lq_prep.h", set(bench.TRAFFIC_SOURCES) - {"sign_fp6_kernel"}),
                                            ("lq_fp6_mma.h", {"sign_fp6_kernel"})])
def test_a_header_that_a_kernel_includes_counts(tree, header, kernels):
    """Through another header too (the preparation's file names lq_prep.h alone)."""
    before = {k: bench.kernel_sources_hash(k) for k in bench.TRAFFIC_SOURCES}
    (tree / header).write_text((tree / header).read_text() + "// more\n")
    assert {k for k in before if bench.kernel_sources_hash(k) != before[k]} == kernels
