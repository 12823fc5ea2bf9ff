"""A stored DRAM-traffic figure outlives changes of sources that its kernel is not made from."""
import json
import os

import pytest

import bench


@pytest.fixture
def tree(tmp_path):
    csrc = tmp_path / "step_flow_map_b200" / "csrc"
    csrc.mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "flashmap.h").write_text("int api;")
    for f, text in {
            "base.cuh": "int base;", "mine.cuh": '#include "base.cuh"\n__global__ void __launch_bounds__(64, 1) k_mine(int a) {}',
            "unit.cu": '#include "flashmap.h"\n#include "mine.cuh"\n#include "other.cuh"\nvoid launch();',
            "other.cuh": '#include "base.cuh"\n__global__ void k_mine_too() {}', "far.cu": '#include "far.cuh"',
            "far.cuh": '#include "base.cuh"\n// k_mine(\n__global__ void k_far() {}'}.items():
        (csrc / f).write_text(text)
    p = tmp_path / "profiles" / "traffic.txt"
    p.parent.mkdir()
    p.write_text(json.dumps({"k_mine": {"wl": {"dram_bytes_per_launch": 7,
                                               "source_sha1": bench.source_sha1(str(tmp_path), "k_mine")}}}))
    return tmp_path


def stored(tree):
    return bench.stored_traffic("k_mine", "wl", root=str(tree))


@pytest.mark.parametrize("f,kept", [("base.cuh", False), ("mine.cuh", False), ("unit.cu", False), ("other.cuh", True),
                                    ("far.cu", True), ("far.cuh", True), ("../../include/flashmap.h", True)])
def test_a_change_counts_where_the_kernel_is_made_of_it(tree, f, kept):
    assert stored(tree) == 7
    p = tree / "step_flow_map_b200" / "csrc" / f
    p.write_text(p.read_text() + "\n// a comment\n")
    assert stored(tree) == 7
    p.write_text(p.read_text() + "int more;")
    assert stored(tree) == (7 if kept else None)


def test_a_new_file_counts_only_if_it_is_included(tree):
    csrc = tree / "step_flow_map_b200" / "csrc"
    (csrc / "new.cuh").write_text("int n;")
    (csrc / "new.cu").write_text('#include "new.cuh"')
    assert stored(tree) == 7
    (csrc / "base.cuh").write_text('#include "new.cuh"\nint base;')
    assert stored(tree) is None


def test_a_kernel_that_no_file_defines_is_made_of_everything(tree):
    assert bench.source_sha1(str(tree), "k_none") == bench.source_sha1(str(tree))
    assert bench.source_sha1(str(tree), "k_mine") != bench.source_sha1(str(tree))


def test_the_persistent_pass_is_not_made_of_the_cache_kernels():
    csrc = os.path.join(bench.ROOT, "step_flow_map_b200", "csrc")
    files = [os.path.basename(f) for f in bench._included(os.path.join(csrc, "fm_dit.cuh"), {})]
    assert "fm_dit.cuh" in files and "fm_tc.cuh" in files
    assert not any(f.startswith("fm_cache") for f in files)
    assert bench.source_sha1(kernel="k_dit_persistent") != bench.source_sha1()
