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


def test_selftest_of_the_waits_refuses():
    """What moe_grouped_mm_w4 refuses, a missing status and limits out of range,
    before any CUDA call."""
    import ctypes

    from expanded_layout_expert_gb300 import _capi, build
    build.build()
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 255) // 256 * 256

    def call(x=p, N=64, Kd=128, most=8, out=p + 1024, limit=1000, status=p):
        return _capi.load().moe_selftest_w4_wait(x, Kd, p, p, None, p, p, 2, N, Kd, 8, most, out, N, limit, 0, 0,
                                                 status, None)

    for kw, text in ((dict(x=None), "non-null"), (dict(N=60), "multiple of 8"), (dict(Kd=64), "Kd of the group"),
                     (dict(most=9), "max_rows"), (dict(out=p), "out must not be x"), (dict(status=None), "null status"),
                     (dict(limit=0), "limit"), (dict(limit=1 << 33), "limit")):
        assert call(**kw) == _capi.MOE_ERR_INVALID_ARG
        assert text in _capi.load().moe_last_error_string().decode(), kw


def test_what_is_under_way_is_waited_for_after_a_wait_gave_up():
    """Products by the lane that issued them, copies by what was asked for: the
    loop's own count goes on without asking."""
    text = kernel()
    load = block(text, text.index("auto load ="))
    asked = load.index("full[kStages + stage] = static_cast<uint32_t>(b - b0 + 1);")
    assert asked < load.index("mbar_arrive_expect_tx(")
    drain = block(text, text.index("if (stop)"))
    assert "to_load" not in drain and "asked" not in drain
    issue = re.search(r"if \((\(warp & 3\) == 0) && elect_one\(\)\) \{\s*tc_fence_after\(\);", text).group(1)
    assert re.search(re.escape(f"if ({issue} && elect_one()) {{") + r"\s*tc_commit\(&done\[half\]\);\s*"
                     r"drain_wait\(&done\[half\], 0\);", drain)
    assert "full[kStages + s]" in drain
