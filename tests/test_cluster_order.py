"""Order between the thread blocks of a cluster, read from the sources: what a
missing barrier or a barrier of too small a scope does depends on timing, so
no run can show it."""
import os
import re

import pytest

from rank_sum_residual_gb300 import _build

# accesses to another block's shared memory
REMOTE = r"map_shared_rank\(|st_dsmem_f32\(|map_rank\("
# a cluster barrier's waiting half
BARRIER = r"cluster\.sync\(\)|cluster_sync\(\)|cluster_wait_acquire\(\)"


def source(name):
    """A source file without its comments."""
    with open(os.path.join(_build.CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels(text):
    """Name and body of every kernel that a source file defines."""
    for m in re.finditer(r"__global__", text):
        name = re.compile(r"(\w+)\s*\((?=const)").search(text, m.end())
        start = at = text.index("{", name.end())
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
            if depth == 0:
                break
        yield name.group(1), text[start:at]


@pytest.mark.parametrize("name", ["farn_kernels.cuh", "farn_route.cu", "farn_product_tc.cuh"])
def test_blocks_have_started_before_their_memory_is_touched(name):
    """A block's shared memory may be accessed by others of its cluster only
    once it is known to run: a cluster barrier comes first."""
    seen = 0
    for kernel, body in kernels(source(name)):
        first = re.search(REMOTE, body)
        if first is None:
            continue
        seen += 1
        assert re.search(BARRIER, body[:first.start()]), kernel
    assert seen
