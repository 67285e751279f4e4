"""bench.py quotes DRAM traffic of the training kernels only while their sources are those of the capture."""

import os

from conftest import ROOT


def test_other_calls_stay_out_of_the_hashed_sources():
    """A declaration of the rotary or draft-tree calls in a file that the hash covers would void every quoted figure."""
    import bench
    files = {f for names in bench._KERNEL_SOURCES.values() for f in names} | {"merge.cu", "common.cuh", "splitkv_internal.h"}
    for name in sorted(files):
        with open(os.path.join(ROOT, "context_block_sparse_b200", "csrc", name)) as f:
            text = f.read().lower()
        for word in ("page_map", "rope", "tree_", "tree::", "paged"):
            assert word not in text, f"{name}: {word}"
