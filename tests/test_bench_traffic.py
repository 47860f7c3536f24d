"""The bench reports recorded DRAM traffic only on the kernel sources that the counters were taken on."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = os.path.join(ROOT, "deepseek_v4_compressed_csa_gb300", "csrc")


@pytest.fixture
def sources(tmp_path):
    shutil.copytree(CSRC, tmp_path / "csrc")
    return tmp_path / "csrc"


def touch(d, name):
    with open(d / name, "a") as f:
        f.write("\n// another line\n")


@pytest.mark.parametrize("name", ["tc_attend_decode.cu", "tc_project.cu", "compress.cu", "tc_indexer.cu", "tc_attend_prefill.cu",
                                  "indexer.cu", "common.cuh", "tc.cuh", "kernels.h", "fp8_row.cuh", "tree.cuh"])
def test_a_source_of_the_counted_kernels_changes_the_hash(sources, name):
    before = bench.csrc_digest(str(sources))
    touch(sources, name)
    assert bench.csrc_digest(str(sources)) != before


@pytest.mark.parametrize("name", ["tc_paged_attend.cu", "paged_attend.cu", "paged.cuh", "add_norm.cu", "checks.c", "tree_topk.cu"])
def test_other_sources_do_not(sources, name):
    before = bench.csrc_digest(str(sources))
    touch(sources, name)
    assert bench.csrc_digest(str(sources)) == before


def test_every_unit_that_defines_a_counted_kernel_is_hashed():
    """The kernels that the profile's table counts are defined in units of the hash."""
    import re
    text = open(os.path.join(ROOT, bench.TRAFFIC["profile"])).read()
    counted = {n for line in text.splitlines() if line.startswith("| k_") for n in re.findall(r"\bk_[a-z0-9_]+", line.split("|")[1])}
    assert len(counted) > 10
    for name in counted:
        units = [f for f in os.listdir(CSRC) if f.endswith(".cu") and
                 re.search(r"__global__[^;{]*\b%s\s*\(" % name, open(os.path.join(CSRC, f)).read())]
        assert units and set(units) <= set(bench.TRAFFIC_UNITS), (name, units)


def test_traffic_is_reported_on_the_recorded_sources_alone(monkeypatch):
    key = "decode_layer_step_bytes"
    monkeypatch.setitem(bench.TRAFFIC, "csrc_sha256", bench.csrc_digest())
    assert bench._traffic(key, 2) == 2 * bench.TRAFFIC[key]
    monkeypatch.setitem(bench.TRAFFIC, "csrc_sha256", "0" * 16)
    assert bench._traffic(key, 2) is None
