"""Rules of the kernels' sources that a run on a GPU would show only by chance."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_06_gb300", "csrc")


def test_kernels_that_start_early_read_their_arguments_by_plain_loads():
    """A launch with programmatic serialization lives while the kernel before it still
    writes: a read-only load may be moved ahead of the wait and may be stale."""
    files = [f for f in glob.glob(os.path.join(CSRC, "*.cu")) if "launch_early(" in open(f).read()]
    assert {os.path.basename(f) for f in files} >= {"rope.cu", "tree.cu", "tree_commit.cu"}
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        assert "griddep_wait()" in code, f
        for word in ("__ldg", "__restrict__", "ld.global.nc"):
            assert word not in code, (f, word)
