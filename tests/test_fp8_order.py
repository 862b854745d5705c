"""Order between the thread blocks of a pair and of a split row in the FP8
products, read from the sources as in test_cluster_order."""
import re

from test_cluster_order import BARRIER, REMOTE, asm_statements, kernels, source

SOURCE = "farn_fp8_product.cuh"
# how the pair waits on each of its barriers: tensor memory alone is handed over
# on acc_*, which the tcgen05 fences order; both blocks' copies and products
# arrive on the ring's; the factors stay within a block
PAIR = {"afull": "kTensor", "aempty": "kTensor", "full": "kCluster", "empty": "kCluster",
        "sfull": "kOwn", "sempty": "kOwn"}


def bodies():
    return dict(kernels(source(SOURCE)))


def test_blocks_have_started_before_their_memory_is_touched():
    seen = 0
    for name, body in bodies().items():
        first = re.search(REMOTE, body)
        if first is not None:
            seen += 1
            assert re.search(BARRIER, body[:first.start()]), name
    assert seen == 2


def waits(body):
    return re.findall(r"f8_(?:look|wait|answer)<(\w+)>\(\s*(?:\w+,\s*)?m\.(\w+)", body)


def test_waits_say_what_they_order():
    found = waits(bodies()["farn_fp8_pair_kernel"])
    assert {bar for _, bar in found} == set(PAIR)
    for kind, bar in found:
        assert kind == PAIR[bar], bar
    one = bodies()["farn_fp8_one_kernel"]
    assert waits(one) and all(kind == "kOwn" for kind, _ in waits(one))
    # the parts of a split row are ordinary memory of other blocks
    assert len(re.findall(r"tc_wait_warp<true>\(part_(?:full|empty)\b", one)) == 2
    assert len(re.findall(r"tc::mbar_arrive_cluster\(tc::map_rank\(part_(?:full|empty)", one)) == 2


def test_relaxed_arrivals_hand_over_tensor_memory_only():
    text = source(SOURCE)
    relaxed = [c for c in asm_statements(text) if "arrive.relaxed" in c]
    assert len(relaxed) == 1 and ".relaxed.cluster.shared::cluster" in relaxed[0]
    calls = [m.start() for m in re.finditer(r"arrive_relaxed\((?!uint32_t)", text)]
    assert len(calls) == 1
    before = text[:calls[0]]
    # behind the reads, and the fence that orders them
    assert before.rindex("fence_before()") > before.rindex("tmem_ld_wait()")
    for m in re.finditer(r"f8_(?:wait|answer)<kTensor>", bodies()["farn_fp8_pair_kernel"]):
        after = bodies()["farn_fp8_pair_kernel"][m.end():]
        assert after.index("fence_after()") < min(
            after.find(x) % (1 << 30) for x in ("tmem_ld32(", "mma_fp8<"))
