"""Instructions of the 16-bit grouped products that want a whole warp at them
(their .aligned forms), in places that lanes reach by different branches: the
lanes are made to meet first. Read from the sources, since a warp that happens
to be together anyway shows nothing."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "expanded_layout_expert_gb300", "csrc")
SOURCES = ("mm16.cuh", "grouped_mm16.cu", "grouped_mm16_few.cu")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def function_body(text, at):
    """The innermost function-level block (column 0 to column 0) around `at`."""
    return text[text.rfind("\n}", 0, at) + 1:at]


def test_cluster_barriers_and_tmem_release():
    seen = 0
    for name in SOURCES:
        text = code(name)
        for m in re.finditer(r"barrier\.cluster\.arrive[^;]*\.aligned|tcgen05\.dealloc|tmem_dealloc\(tmem", text):
            before = function_body(text, m.start())
            # `tmem_dealloc(taddr, ...)` of one CTA's form stands in a function that has met already
            assert "__syncwarp();" in before[-500:], (name, m.group(0))
            seen += 1
    assert seen >= 3   # cluster_sync, the pair's release, the few-rows form's


def test_accumulator_reads_after_stores_of_single_lanes():
    """A TMEM load is warp-wide; the loop before it stores what its lane has."""
    seen = 0
    for name in SOURCES[1:]:
        text = code(name)
        for m in re.finditer(r"\btc_ld32_wait\(", text):
            assert "__syncwarp();" in text[max(0, m.start() - 120):m.start()], name
            seen += 1
    assert seen == 2
