"""Counters are dropped once any source of their kernel changes (CPU)."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """bench.py on a copy of the kernel sources."""
    sys.path.insert(0, ROOT)
    import bench
    shutil.copytree(os.path.join(ROOT, "moe_expert_load_amd", "csrc"),
                    tmp_path / "moe_expert_load_amd" / "csrc")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return bench, tmp_path / "moe_expert_load_amd" / "csrc"


def digests(bench):
    return {k: bench.source_digest(k) for k in bench.KERNEL_SOURCES}


@pytest.mark.parametrize("header,users", [("q8.hpp", {"gemm.hip"}),
                                          ("common.hpp", {"gemm.hip", "swiglu.hip", "copy.hip", "plan.hip"}),
                                          ("gemm.hip", {"gemm.hip"}), ("router.hpp", set())])
def test_headers_of_a_kernel_count(tree, header, users):
    bench, csrc = tree
    before = digests(bench)
    text = (csrc / header).read_text()
    (csrc / header).write_text(text + "// a comment\n")
    assert digests(bench) == before
    (csrc / header).write_text(text + "static int more;\n")
    changed = {k for k, v in digests(bench).items() if v != before[k]}
    assert changed == {k for k, src in bench.KERNEL_SOURCES.items() if os.path.basename(src) in users}


def test_every_include_is_followed(tree):
    bench, _ = tree
    names = [os.path.basename(p) for p in bench.kernel_sources("k_wgrad")]
    assert names[0] == "gemm.hip" and {"common.hpp", "host.hpp", "q8.hpp"} <= set(names)
    assert len(names) == len(set(names))
