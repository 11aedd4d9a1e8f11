"""The DRAM traffic that bench.py reports comes from profiles of the kernel
sources at hand: the hash that ties them covers every local file the LM head
includes, and the committed profiles carry it."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "block_draft_selection_b200", "csrc")
WORKLOADS = ["throughput", "qwen3-4b-bs1", "qwen3-4b-batched", "27b-class"]


def _read(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_hash_covers_what_the_kernel_includes():
    files = bench.kernel_sources()
    assert files[0] == "lmhead_topk.cu" and len(set(files)) == len(files)
    for f in files:
        for inc in re.findall(r'#include "([^"]+)"', _read(f)):
            assert inc in files or inc == "../../include/dflash.h", (f, inc)
    assert "host_util.cuh" in files and "common.cuh" in files


def test_a_change_in_any_of_them_changes_the_hash(tmp_path, monkeypatch):
    for f in bench.kernel_sources():
        (tmp_path / f).write_text(_read(f))
    monkeypatch.setattr(bench, "CSRC", str(tmp_path))
    before = bench.kernel_source_hash()
    for f in bench.kernel_sources():
        text = (tmp_path / f).read_text()
        (tmp_path / f).write_text(text + "// another line\n")
        assert bench.kernel_source_hash() != before, f
        (tmp_path / f).write_text(text)
    assert bench.kernel_source_hash() == before


@pytest.mark.parametrize("workload", WORKLOADS)
def test_committed_profiles_are_of_these_sources(workload):
    traffic = bench.profiled_traffic(workload)
    assert traffic is not None, "profiles/lmhead_topk_%s.md was taken on other sources: take it again" % workload
    w = bench.syn.workload(workload)
    assert traffic >= 2 * w.V * w.d          # W is read at least once
