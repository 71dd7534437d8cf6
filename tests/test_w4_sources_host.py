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


def constants(name, *wanted):
    """The source's one-line constants and the named functions, as C++."""
    text = code(name)
    lines = re.findall(r"^constexpr int \w+ = [\w *+/()]+;", text, re.M)
    for f in wanted:
        m = re.search(rf"^(?:constexpr )?int {f}\([^)]*\) ", text, re.M)
        lines.append(m.group(0) + block(text, m.end() - 1))
    return "\n".join(lines)


def test_ctas_of_an_sm_find_room_in_tensor_memory(tmp_path):
    """What may lie on an SM together, by shared memory alone, holds at most 512
    columns: an allocation that waits has no limit, and CTAs of clusters that wait
    for one another would then wait for ever."""
    import itertools
    import subprocess
    launch = code(NAME)[code(NAME).index("int launch("):]
    f = re.search(r"constexpr int kSmem = (\w+)\(kGroup, kR\);", launch).group(1)
    wanted = ["step_k", "stage_bytes", "stages_for", "ring_bytes"] + ([f] if f != "ring_bytes" else [])
    src = tmp_path / "smem.cpp"
    src.write_text(f"""#include <cstdio>
namespace w4 {{ {constants(NAME, *wanted)} }}
namespace few {{ {constants("grouped_mm16_few.cu", "stages_for", "ring_bytes")} }}
int main() {{
  for (int g = 32; g <= 128; g *= 2)
    for (int R = 16; R <= (g == 32 ? 32 : 64); R += 16)
      std::printf("%d %d\\n", w4::{f}(g, R), w4::kTmemCols);
  for (int R = 16; R <= 128; R *= 2) std::printf("%d %d\\n", few::ring_bytes(R), R < 32 ? 32 : R);
}}
""")
    exe = tmp_path / "smem"
    subprocess.run(["g++", "-std=c++17", "-w", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    ctas = sorted({tuple(map(int, line.split())) for line in out.splitlines()})
    assert len(ctas) >= 8 and {c for _, c in ctas} == {32, 64, 128, 256}
    for n in (2, 3, 4):
        for some in itertools.combinations_with_replacement(ctas, n):
            if sum(b + 1024 for b, _ in some) <= 228 * 1024:   # 1 KB a CTA is the system's
                assert sum(c for _, c in some) <= 512, some
