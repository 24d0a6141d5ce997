"""The bench line's HBM traffic: the committed counter record belongs to the sources that its kernels are built from."""
import os
import re
import shutil

import pytest

import bench

CSRC = os.path.join("post_quantization_03_amd", "csrc")


def test_committed_traffic_is_reported():
    assert bench.measured_traffic("hg_sqrt") > 10 ** 10
    assert bench.measured_traffic("quantize") is None      # no record


@pytest.mark.parametrize("source,ages", [("norm.hip", False), ("tile.h", False), ("sweep.hip", False), ("gj.hip", True), ("dense.hip", True),
                                         ("kq_internal.h", True)])
def test_only_the_phase_s_sources_age_its_record(tmp_path, monkeypatch, source, ages):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    shutil.copytree(os.path.join(bench.ROOT, "profiles"), tmp_path / "profiles")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.measured_traffic("hg_sqrt")
    assert before
    with open(tmp_path / CSRC / source, "a") as f:
        f.write("// changed\n")
    assert bench.measured_traffic("hg_sqrt") == (None if ages else before)


def test_square_root_s_kernels_are_in_its_sources():
    """Every kernel that the square root's file launches or that its products come from is defined in the listed files."""
    text = {f: open(os.path.join(bench.ROOT, CSRC, f)).read() for f in bench.PHASE_SOURCES["hg_sqrt"]}
    kernels = set(re.findall(r"__global__[^{;]*?\b(\w+_kernel)\(", "".join(text.values())))
    launched = set(re.findall(r"hipLaunchKernelGGL\(\(*(\w+_kernel)", "".join(text.values())))
    assert launched and launched <= kernels, launched - kernels
    assert set(re.findall(r'#include "([\w.]+)"', "".join(text.values()))) <= set(text)
