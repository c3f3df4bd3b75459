"""The hand-over of the rows' references between the two sets of warps of attend_tc_kernel, in every order in which warps can
run: a model of its barriers, which know a phase by its parity only, and the order of waits in the kernel's source."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WARPS = 2  # of a set; the kernel's eight do the same


def program(me: int, segments, second_waits_first: bool):
    """What a warp of set `me` does, tile by tile: ("wait", set, phase), ("arrive",) at its own set's barrier, ("sync",)."""
    ops, gt = [], 0
    for tiles in segments:
        for j in range(tiles):
            if gt % 2 == me:
                before, behind = ("wait", 1 - me, (gt - 1) // 2), ("wait", 1 - me, (gt + 1) // 2)
                if j >= 2:
                    ops += [before, ("arrive",)]
                elif j == 1:
                    ops += [before, ("arrive",)] if second_waits_first else [("arrive",), before]
                else:
                    ops += [("arrive",)] + ([behind] if tiles > 1 else [])
            gt += 1
        ops.append(("sync",))
    return ops


def explore(segments, second_waits_first: bool):
    """Walks through every state that some order of the warps reaches.  "": all orders end; else what goes wrong."""
    programs = [program(s, segments, second_waits_first) for s in (0, 1) for _ in range(WARPS)]
    start = ((0,) * len(programs), (0, 0), (0, 0))  # each warp's place; the barriers' phases; arrivals in them
    seen, todo = {start}, [start]
    while todo:
        at, phase, arrived = todo.pop()
        if all(i == len(p) for i, p in zip(at, programs)):
            continue
        found = []
        if all(i < len(p) and p[i] == ("sync",) for i, p in zip(at, programs)):
            found.append((tuple(i + 1 for i in at), phase, arrived))
        for w, (i, p) in enumerate(zip(at, programs)):
            if i == len(p) or p[i] == ("sync",):
                continue
            ph, ar = list(phase), list(arrived)
            if p[i][0] == "wait":
                if phase[p[i][1]] % 2 == p[i][2] % 2:
                    continue  # the parity says that the phase is not over
                if phase[p[i][1]] <= p[i][2]:
                    return "a wait passes before its phase is over"
            else:
                s = w // WARPS
                ar[s] += 1
                if ar[s] == WARPS:
                    ph[s], ar[s] = ph[s] + 1, 0
            found.append((at[:w] + (i + 1,) + at[w + 1:], tuple(ph), tuple(ar)))
        if not found:
            return "warps wait for good"
        for state in found:
            if state not in seen:
                seen.add(state)
                todo.append(state)
    return ""


@pytest.mark.parametrize("segments", [(1,), (2,), (3,), (7,), (1, 1, 1), (1, 2, 3), (3, 3), (5, 1, 4), (2, 2, 2), (4, 1, 1, 6)])
def test_every_order_of_the_warps_ends(segments):
    assert explore(segments, second_waits_first=True) == ""


def test_a_second_tile_that_arrives_first_can_be_overtaken():
    """Its set has arrived, the other one takes the next two phases' parity away from a warp that has yet to look."""
    assert explore((3,), second_waits_first=False) == "warps wait for good"


def test_the_kernel_waits_in_that_order():
    with open(os.path.join(ROOT, "gdn_speculative_tree_gb300", "csrc", "attend_tc.cu")) as f:
        block = re.search(r"if \(start\) \{(.*?)\n        \} else \{", f.read(), re.S).group(1)
    waits = [m.start() for m in re.finditer(r"wait_warp\(rs, &cs\.mdone\[set \^ 1\]", block)]
    arrive = block.index("warp_arrive(&cs.mdone[set])")
    assert len(waits) == 2 and waits[0] < arrive < waits[1]
    assert re.search(r"if \(j != t0\) wait_warp\(rs, &cs\.mdone\[set \^ 1\], \(\(gt - 1\) >> 1\) & 1\)", block)
    assert re.search(r"if \(j == t0\) wait_warp\(rs, &cs\.mdone\[set \^ 1\], \(\(gt \+ 1\) >> 1\) & 1\)", block)
