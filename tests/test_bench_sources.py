"""bench.py's stored counters go with the sources of the kernels they were taken
of: they stay valid while other sources change, and no longer."""
import os
import shutil

import pytest

import bench


def test_stored_traffic_is_of_the_present_kernels():
    sha = bench.kernel_sources_sha()
    for name in [bench.HEADLINE] + bench.NESTED:
        traffic, info = bench.read_traffic(name, sha)
        assert isinstance(traffic, int) and traffic > 0, (name, info)


@pytest.mark.parametrize("source,matters", [("msd_prefill.hip", True), ("msd_device.hpp", True), ("mx_gemv.hip", False),
                                            ("mx_another.hip", False), ("msd_api.cpp", False)])
def test_only_the_kernels_sources_matter(monkeypatch, tmp_path, source, matters):
    before = bench.kernel_sources_sha()
    csrc = os.path.join("weight_only_quantized_msd_amd", "csrc")
    shutil.copytree(os.path.join(bench.ROOT, csrc), tmp_path / csrc)
    with open(tmp_path / csrc / source, "a") as f:
        f.write("// changed\n")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert (bench.kernel_sources_sha() != before) == matters
