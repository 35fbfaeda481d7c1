"""What the linear-attention kernels' source has to say and no run on one compiler can show (CPU)."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_decode_weight_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_number_that_a_call_gives_is_read_in_a_later_statement():
    """cut(chunks, n) gives n; the order of a call's arguments is the compiler's."""
    statements = [s for s in re.split(r"[;{}]", source("linear_prompt.cu")) if re.search(r"\bcut\([^()]*\bn\)", s)]
    assert len(statements) >= 2
    for s in statements:
        assert len(re.findall(r"\bn\b", s)) == 1, s.strip()


def test_the_warps_of_a_group_change_their_registers_by_one_instruction():
    """setmaxnreg is one instruction of all four warps of a group: none stands where a condition on the warp lets fewer of them through."""
    s = source("linear_prompt.cu")
    calls = [m.start() for m in re.finditer(r"\b(fewer|more)_registers<\d+>\(\)", s) if "asm" not in s[m.start():m.start() + 60]]
    assert len(calls) == 5
    for at in calls:
        depth = 0
        for m in reversed(list(re.finditer(r"[{}]", s[:at]))):
            depth += 1 if m.group() == "}" else -1
            if depth < 0:                                     # the block that the call stands in
                head = s[s.rfind("\n", 0, m.start()):m.start()]
                break
        assert "warp ==" not in head and all(int(n) % 4 == 0 for n in re.findall(r"warp < (\d+)", head)), head
