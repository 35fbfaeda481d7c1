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


def ends(start, moves):
    """The states that can be reached from `start` and from which nothing moves any more."""
    seen, todo, last = {start}, [start], []
    while todo:
        s = todo.pop()
        after = list(moves(s))
        last += [] if after else [s]
        for t in after:
            if t not in seen:
                seen.add(t)
                todo.append(t)
    return last


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


# ------------------------------------------------------- every warp that waits for a copy sees its phase


def keys_first(count):
    """The units of an item: K0 K1 V0 K2 V1 ... with their tiles."""
    order = [("K", 0)]
    for i in range(count):
        order += [("K", i + 1)] if i + 1 < count else []
        order += [("V", i)]
    return order


def stuck(scores_wait, slots, count):
    """Whether the ring of 16-bit tiles can come to a halt: a copying warp, the warp of the products (which frees a slot) and
    two helper warps, that wait for every unit's copy and then arrive. A barrier is the number of its completed
    phases, and a wait for phase n by parity returns while that is n + 1, n + 3, ..."""
    order = keys_first(count)
    place = {u: n for n, u in enumerate(order)}
    products = [("K", 0)] + ([("K", 1)] if count > 1 else [])
    for i in range(count):
        products += [("V", i)] + ([("K", i + 2)] if i + 2 < count else [])
    n = len(order)
    assert sorted(products) == sorted(order)

    def over(done, phase):
        return done > phase and (done - phase) % 2 == 1

    # asked, arrived: copies; freed per slot; place of the products; places of the helpers
    def moves(s):
        asked, arrived, used, helpers = s
        freed = [sum(1 for u in products[:used] if place[u] % slots == x) for x in range(slots)]
        full = [sum(1 for u in range(arrived) if u % slots == x) for x in range(slots)]
        clean = [min(sum(1 for u in range(h) if u % slots == x) for h in helpers) for x in range(slots)]
        if asked < n and freed[asked % slots] >= asked // slots:
            yield asked + 1, arrived, used, helpers
        if arrived < asked:
            yield asked, arrived + 1, used, helpers
        if used < n:
            u = place[products[used]]
            done = full if products[used][0] == "K" and scores_wait == "full" else clean
            if over(done[u % slots], u // slots):
                yield asked, arrived, used + 1, helpers
        for j, h in enumerate(helpers):
            if h < n and over(full[h % slots], h // slots):
                yield asked, arrived, used, helpers[:j] + (h + 1,) + helpers[j + 1:]

    return any(s != (n, n, n, (n, n)) for s in ends((0, 0, 0, (0, 0)), moves))


@pytest.mark.parametrize("slots,count", [(3, 6), (4, 7), (5, 8)])
def test_ring_of_tiles_cannot_come_to_a_halt(slots, count):
    """The products wait for the helpers' arrival for keys as for values; waiting for the copy alone lets a slot be
    filled again before a helper has seen that its last copy is there."""
    assert stuck("full", slots, count) and not stuck("clean", slots, count)
    scores = re.search(r"auto scores = \[&\]\(int i\) \{(.*?)tc_fence_after", source("tree_attention.cu"), re.S).group(1)
    assert re.findall(r"wait\(([^;]*?) \+ 8 \* at", scores) == ["sm.clean"]
