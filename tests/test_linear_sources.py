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
