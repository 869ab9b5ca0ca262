"""bench.py's hash of a kernel's sources covers every device header the kernel is built from, so that a change in any of
them voids the DRAM figures captured before it (no GPU needed)."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "routed_expert_ffn_softmax_gb300", "csrc")


def device_headers(name, seen=None):
    """The .cuh files that a source includes, directly or through others."""
    seen = set() if seen is None else seen
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        for h in re.findall(r'^#include "(\w+\.cuh)"', f.read(), flags=re.M):
            if h not in seen:
                seen.add(h)
                device_headers(h, seen)
    return seen


@pytest.mark.parametrize("sources", ["EXPERT_SOURCES", "DECODE_SOURCES", "ATTN_SOURCES"])
def test_the_hash_covers_the_headers(sources):
    names = getattr(bench, sources)
    for name in names:
        assert device_headers(name) <= set(names), name
    assert any(device_headers(name) for name in names)
