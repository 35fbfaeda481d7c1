"""The rings of asynchronous copies as sets of roles, all of whose orders are tried (CPU).

A role is a list of steps; a step is (when it may happen, what it does) over a small state. What a kernel does is
read from its source: which barriers a role waits for, and under which condition a block waits for its copies."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_decode_weight_gb300", "csrc")


def source(name):
    """A kernel's source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# ------------------------------------------------------------- a block does not end before its copies


def copies_left(always, copies=2):
    """Whether a block can end while a copy is in flight. Its copying warp requests all copies (they fit into free slots),
    then waits for them, always or where it sees that the block gave up; the other warp waits for each copy, and gives
    up at any time."""
    # asked, arrived, place of the copying warp (0 requests, 1 waits for its copies, 2 over), of the other (copy it waits for, or over), given up
    def moves(s):
        asked, arrived, warp, other, dead = s
        if arrived < asked:
            yield asked, arrived + 1, warp, other, dead
        if warp == 0:
            if asked < copies and not dead:
                yield asked + 1, arrived, 0, other, dead
            else:
                yield asked, arrived, 1 if always or dead else 2, other, dead
        elif warp == 1 and arrived == asked:
            yield asked, arrived, 2, other, dead
        if other < copies:
            if arrived > other or dead:
                yield asked, arrived, warp, other + 1, dead
            if not dead:
                yield asked, arrived, warp, other, True

    todo, seen = [(0, 0, 0, 0, False)], set()
    while todo:
        s = todo.pop()
        if s in seen:
            continue
        seen.add(s)
        if s[2] == 2 and s[3] == copies and s[1] < s[0]:
            return True
        todo += moves(s)
    return False


def test_a_block_that_gives_up_late_needs_an_unconditional_wait():
    assert copies_left(always=False) and not copies_left(always=True)


@pytest.mark.parametrize("name,drain", [("tree_attention.cu", r"mbar_drain\(sm\.full"), ("tree_attention_rows.cu", r"mbar_drain_inline\(full"),
                                        ("w4_tensor.cu", r"mbar_drain\(bar\(L::kFull")])
def test_copying_warps_wait_for_their_copies_unconditionally(name, drain):
    lines = [l.strip() for l in source(name).splitlines() if l.strip()]
    at = [i for i, l in enumerate(lines) if re.search(drain, l)]
    assert len(at) == 1 and lines[at[0]].startswith("for (")
    before = lines[at[0] - 1]
    assert not re.match(r"if \(.*(dead|lost)", before), before
