"""The ncu summary of the rows kernel over pages carries a digest of its sources, comments and layout left out."""
import hashlib
import os
import re

import pytest

import bench

SOURCES = ["rows_kernel.cuh", "rows_plan.cuh", "rows_ptx.cuh", "paged.h"]
CSRC = os.path.join(bench.ROOT, "gqa_decode_blackwell_gb300", "csrc")


def tree_source_digest():
    h = hashlib.sha256()
    for name in SOURCES:
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            h.update(bench._code_only(f.read()).encode())
    return h.hexdigest()[:16]


def test_the_summary_is_of_the_present_kernel():
    """A kernel that is not profiled yet is a skip, as for the other summaries."""
    with open(os.path.join(bench.PROFILES, "rows_kernel_tree.md"), encoding="utf-8") as f:
        field = re.search(r"tree_source_sha256: `([0-9a-f]{16})`", f.read())
    assert field is not None
    if field.group(1) != tree_source_digest():
        pytest.skip(f"rows kernel code {tree_source_digest()} differs from its ncu summary: capture it again")
