"""Prompt attention's bounded waits have one answer per warp (read from the source: a lane that went on alone would wait
for the others in its next warp-wide instruction, and the kernel would not end)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_kv_cache_kvarn_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def body(text, head):
    """From the head's opening brace to the closing one."""
    start = text.index("{", text.index(head))
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(head)


def test_a_warps_wait_votes_on_both_ends():
    wait = body(source("kvarn_common.cuh"), "bool mbar_wait_warp(")
    assert "if (__all_sync(0xffffffffu, done)) return true;" in wait
    ends = re.findall(r"if \((.*)\) (?:return false|break);", wait)
    assert len(ends) == 2 and all(e.startswith("__any_sync(0xffffffffu, ") for e in ends)


def test_only_votes_follow_the_waits_of_lanes():
    text = source("prompt_attn.cu")
    assert "mbar_wait_warp(" in body(text, "bool wait_for(") and "mbar_wait_warp(" in body(text, "bool wait_unit(")
    lines = text.splitlines()
    for i, line in enumerate(lines):
        if "lane_wait_for" not in line or "bool lane_wait_for(" in line:
            continue
        if "lane_wait_for<true>" in line or "const bool got = lane_wait_for" in line:  # drain, my_turn
            continue
        assert any("__all_sync(0xffffffffu, " in l for l in lines[i:i + 4]), line
    for i, line in enumerate(lines):
        if "my_turn()" in line:
            assert any("__all_sync(0xffffffffu, " in l for l in lines[i:i + 4]), line
