"""The key of the recorded DRAM traffic: the quantizers' and GEMMs' sources and nothing else."""
import json
import os
import re
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_precision_bsq_gb300", "csrc")
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.fixture()
def copy(tmp_path):
    for name in os.listdir(CSRC):
        shutil.copy(os.path.join(CSRC, name), tmp_path / name)
    return tmp_path


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h", ".cpp"))))
def test_only_the_recorded_kernels_sources_change_the_key(copy, name):
    key = bench.kernel_source_hash(str(copy))
    text = (copy / name).read_text()
    (copy / name).write_text(text + "// a comment\n")
    assert bench.kernel_source_hash(str(copy)) == key
    (copy / name).write_text(text + "int more = 1;\n")
    assert (bench.kernel_source_hash(str(copy)) != key) == (name in bench.TRAFFIC_SOURCES)


def test_a_new_source_does_not_change_the_key(copy):
    key = bench.kernel_source_hash(str(copy))
    (copy / "bsq_another.cu").write_text("int more = 1;\n")
    assert bench.kernel_source_hash(str(copy)) == key


def test_the_recorded_kernels_are_in_the_sources_of_the_key():
    code = "".join(open(os.path.join(CSRC, n), encoding="utf-8").read() for n in bench.TRAFFIC_SOURCES)
    with open(bench.TRAFFIC_PATH) as f:
        record = json.load(f)
    for workload in record.values():
        for kernel in workload["kernels"]:
            assert re.search(r"__global__[^;{]*\b%s\(" % re.escape(kernel.split("<")[0]), code, re.S), kernel
