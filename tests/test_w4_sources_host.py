"""What the 4-bit product on tcgen05 has to keep and no run shows: read from its
source."""
import os
import re

from test_warp_convergence_host import CSRC, code, function_body

NAME = "grouped_w4.cu"


def kernel():
    text = code(NAME)
    return text[text.index("grouped_w4_kernel("):text.index("int launch(")]


def block(text, at):
    """The braces that open at or after `at`, with what is between them."""
    a = text.index("{", at)
    depth = 0
    for i in range(a, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[a:i + 1]
    raise ValueError("unbalanced braces")


def test_lanes_meet_before_tensor_memory_is_read_or_written():
    """Loads and stores of tensor memory are warp-wide. One lane issues the
    products and copies of a step before; the test of the barrier after it makes the
    lanes meet, also once a wait has given up."""
    text = kernel()
    expect = block(text, text.index("auto expect ="))
    assert re.match(r"\{\s*const bool there = try_wait\(bar, parity\);", expect)
    source = code(NAME)
    assert re.search(r"return __all_sync\(0xffffffffu, \w+ != 0\);\s*\}$", block(source, source.index("bool try_wait(")))
    sums = list(re.finditer(r"\badd\(\);", text))
    assert len(sums) == 2   # of the loop and after it
    for m in sums:
        assert re.search(r"expect\(d_bar, [^;]*;\s*tc_fence_after\(\);\s*$", text[:m.start()])
    # the values of a step: after the sums, or the wait for the stage
    first = text.index("if (h > 0 || !first)")
    stores = text.index("tc_st16(")
    assert first < text.index("expect(bar, &full[slot]") < stores
    assert text.count("tc_ld16_wait(") == 1 and text.count("tc_st16(") == 1
    for m in re.finditer(r"elect_one\(\)", text[first:stores]):
        raise AssertionError("a lane of its own between the waits and the stores")


def test_cluster_barriers_and_tmem_release():
    text = code(NAME)
    assert "barrier.cluster" not in text   # by cluster_sync alone, which has the lanes meet
    seen = 0
    for m in re.finditer(r"tmem_dealloc\(tmem", text):
        assert "__syncwarp();" in function_body(text, m.start())[-100:]
        seen += 1
    assert seen == 1

