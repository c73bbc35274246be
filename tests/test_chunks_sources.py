"""CPU checks of the sources of the attention over chunks and of what belongs to it: what can only be seen by reading."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_quantized_linear_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def kernels(text):
    """(name, body) of every kernel."""
    for m in re.finditer(r"__global__ void[^{;]*?(\w+)\((?:[^(){};]|\([^()]*\))*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


@pytest.mark.parametrize("name,count", [("attn_chunks_i4.cu", 2), ("attn_steps_i4.cu", 1), ("kv_weights_i4.cu", 2), ("kv_evict_i4.cu", 1)])
def test_kernels_wait_for_what_came_before_them_on_every_path(name, count):
    # they may begin before the kernel in front of them ends: what that one, or one before it, wrote is theirs to read only
    # after a wait of their own
    found = list(kernels(source(name)))
    assert len(found) == count
    for kernel, body in found:
        waits = [m.start() for m in re.finditer(r"grid_dependency_wait\(\);", body)]
        assert len(waits) == 1, kernel
        before = body[:waits[0]]
        assert before.count("{") == before.count("}"), (kernel, "the wait is on one path only")
        assert re.search(r"(^|[;}])\s*$", before), (kernel, "the wait is on one path only")
        # nothing that an argument points to is read before it (the pointers themselves are parameters)
        assert not re.search(r"\ba\.[\w.]+\s*\[|chunk\(|__ldg|tma_load|bulk_load|->", before), kernel


def test_rings_that_groups_use_in_turn_are_asserted_to_go_round_with_them():
    # a group that sees every other phase of a slot's barrier can take an old one for the next: each such ring says why it cannot
    chunks, weights = source("attn_chunks_i4.cu"), source("kv_weights_i4.cu")
    for text, ring in ((chunks, r"kRaw % 2 == 0"), (chunks, r"kSlots % 2 == 0"), (weights, r"kKeySlots % kConv == 0"), (weights, r"2 % kConv == 0"),
                       (weights, r"2 % kSoft == 0")):
        assert re.search(r"static_assert\([^;]*" + ring, text), ring
