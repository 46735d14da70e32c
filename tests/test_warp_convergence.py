"""Warp-collective (.aligned) instructions outside the inner loops: an instruction that needs
all lanes of a warp together stands behind a __syncwarp() in its own wrapper, because callers
reach it after branches and loops in which lanes part. A missing one can hang or fault a GPU,
so this is checked in the source text."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp8_block_scaled_05_gb300", "csrc")
GUARDED = ("barrier.cluster.arrive", "barrier.cluster.wait", "tcgen05.alloc", "tcgen05.dealloc")


def functions():
    """(file, name, body) of every device function that holds an asm statement."""
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"__device__ __forceinline__ \w+ (\w+)\([^{;]*\)\s*\{(.*?)\n\}", text,
                             re.S):
            if "asm" in m[2]:
                yield name, m[1], m[2]


@pytest.mark.parametrize("instruction", GUARDED)
def test_guarded_by_a_syncwarp(instruction):
    found = [(f, n, body) for f, n, body in functions()
             if re.search(re.escape(instruction) + r"[\w.:]*\.aligned", body)]
    assert found, instruction
    for f, n, body in found:
        before = body[:body.index(instruction)]
        assert "__syncwarp()" in before, f"{f}: {n}"


def test_no_bare_cluster_barrier():
    """Cluster barriers are reached through their wrappers alone."""
    for name in sorted(os.listdir(CSRC)):
        if name != "device.cuh":
            assert "barrier.cluster" not in open(os.path.join(CSRC, name)).read(), name
