"""Arrivals on mbarriers that order nothing, read in the sources.  Such an arrival may hand
back tensor memory alone, whose reads tcgen05's own fence has ordered before it; shared memory
that the arriving threads have read is handed back by an arrival that releases, or the
next copy into it may overtake those reads."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "shared_memory_tiled_gb300", "csrc")


def calls():
    for name in sorted(os.listdir(CSRC)):
        lines = open(os.path.join(CSRC, name)).read().split("\n")
        for i, line in enumerate(lines):
            m = re.search(r"ptx::(mbar_arrive_relaxed|mbar_arrive_at)\((.*)\);", line)
            if m:
                yield name, i + 1, m.group(2), "\n".join(lines[max(0, i - 3):i])


def test_arrivals_without_order_hand_back_tensor_memory_only():
    found = list(calls())
    assert len(found) >= 2
    for name, line, barrier, before in found:
        assert re.match(r"sums_empty\b|release\[", barrier), (name, line, barrier)
        assert "tc_fence_before()" in before, (name, line)


def test_release_names_the_barriers_of_tensor_memory():
    text = open(os.path.join(CSRC, "matmul_fp8.cu")).read()
    m = re.search(r"const uint32_t release\[2\] = \{(.*?)\};", text)
    assert m and m.group(1) == "ptx::peer_addr(sums_empty, 0), ptx::peer_addr(sums_empty + 1, 0)"
