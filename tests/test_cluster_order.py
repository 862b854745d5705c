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


def asm_statements(text):
    """The instructions of every asm statement, its string parts joined."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        parts = re.match(r'\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', text[m.end():])
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', parts.group(1)))


def test_arrivals_at_other_blocks_release_to_the_cluster():
    """An arrival on another block's barrier hands over what came before it
    only if it releases at the cluster's scope (without a scope: its own
    block's), itself or by a fence in front of it."""
    seen = 0
    for code in asm_statements(source("farn_tcgen05.cuh")):
        for m in re.finditer(r"mbarrier\.arrive[.\w]*(?:::\w+[.\w]*)*", code):
            name = m.group(0)
            if "shared::cluster" not in name:
                continue
            seen += 1
            if ".release.cluster" in name:
                continue
            assert ".relaxed.cluster" in name, name
            assert re.search(r"fence\.(release|acq_rel)[.\w:]*\.cluster;", code[:m.start()]), name
    assert seen


def test_waits_for_other_blocks_acquire_from_the_cluster():
    """The other half: a wait says whether other blocks arrive on its barrier,
    and one for them acquires at the cluster's scope."""
    waits = [c for c in asm_statements(source("farn_tcgen05.cuh")) if "try_wait" in c]
    assert any(".acquire.cluster" in c for c in waits)
    text = source("farn_product_tc.cuh")
    # how the kernel waits on each of its barriers: always, or in a pair of
    # blocks only, with the cluster's scope
    scope = {"part_full": "true", "part_empty": "true", "full0": "kPair", "empty0": "kPair",
             "sfull0": "kPair", "sempty0": "kPair", "tfull0": "kPair", "tempty0": "kPair"}
    found = set()
    for m in re.finditer(r"tc_wait_warp(?:<(\w+)>)?\(\s*(?!uint32_t)(\w+)", text):
        if m.group(2) in scope:
            assert m.group(1) == scope[m.group(2)], m.group(0)
            found.add(m.group(2))
    assert found == set(scope)
    assert re.search(r"kPair = CG == 2;", text)


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in _build.DEPENDS))
def test_copies_go_to_one_block(name):
    """Operands may lie in any memory that the device can read, so a copy to
    shared memory goes to one block: none is multicast over a cluster."""
    path = next(p for p in _build.DEPENDS if os.path.basename(p) == name)
    for code in asm_statements(source(path)):
        assert not ("cp.async.bulk" in code and "multicast" in code), code
