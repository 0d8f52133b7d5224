"""bench.py's DRAM traffic figures are keyed to hashes of the kernels' sources:
the hashed files are all that those kernels are compiled from (no GPU)."""
import os
import re

import bench

CSRC = "paged_kv_cache_291_gb300/csrc/"
HOST_ONLY = {CSRC + "pkv_internal.h"}  # launch descriptions, no device code


def included(rel, seen):
    with open(os.path.join(bench.ROOT, rel)) as f:
        for name in re.findall(r'#include "([^"]+)"', f.read()):
            path = CSRC + name
            if path not in seen and os.path.exists(os.path.join(bench.ROOT, path)):
                seen.add(path)
                included(path, seen)
    return seen


def test_hashed_sources_hold_every_header():
    for group, files in bench.KERNEL_SOURCES.items():
        needed = set(files)
        for rel in files:
            included(rel, needed)
        assert needed - HOST_ONLY == set(files), group


def test_every_figure_names_its_sources():
    for rec in bench.NCU_TRAFFIC.values():
        assert rec["bytes"] > 0 and rec["sources"] in bench.KERNEL_SOURCES and len(rec["sources_sha"]) == 16
    for group in bench.KERNEL_SOURCES:
        assert len({r["sources_sha"] for r in bench.NCU_TRAFFIC.values() if r["sources"] == group}) == 1
