"""Bounded waits of warps that go on together (CPU only, on the sources).

`mbar_wait` polls a barrier and the CTA's abort flag in each lane by itself.
Where the barrier completes while another warp gives up, a lane that polled
before sees the flag, one that polls after sees the phase: the lanes of a warp
may answer differently.  What follows in a warp that works as one (its
tensor-memory loads, its __syncwarp) is undefined for a part of the lanes and
can wait forever.  So a wait either belongs to a single lane or its answer is
put to the vote of the warp.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp4_fp8_quantization_gb300", "csrc")


def lane_answers(completes_at, aborted_at, polls):
    """What each lane's wait returns: lane i looks at the barrier at time
    polls[i][0], and, if it is not complete, at the flag at polls[i][1], and
    so on in turn."""
    out = []
    for times in polls:
        answer = None
        for i, t in enumerate(times):
            if i % 2 == 0 and t >= completes_at:
                answer = True
            elif i % 2 == 1 and t >= aborted_at:
                answer = False
            if answer is not None:
                break
        out.append(answer)
    return out


def test_lanes_of_one_wait_can_answer_differently():
    polls = [[1, 4, 7, 10], [1, 2, 6, 8], [5, 6, 9, 10]]
    got = lane_answers(completes_at=5, aborted_at=3, polls=polls)
    assert got == [False, True, True]
    vote = [all(got)] * len(got)          # __all_sync: the same for every lane
    assert vote == [False] * 3


def _waits(src):
    """(line, protected) of each mbar_wait call: inside an argument of
    __all_sync, or in a block that a single lane enters."""
    src = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), src)
    found = []
    calls = {m.start() for m in re.finditer(r"\bmbar_wait\s*(<\w+>)?\s*\(", src)}
    open_parens, open_blocks, head = [], [], 0
    for i, ch in enumerate(src):
        if i in calls:
            voted = any(name.endswith("__all_sync") for name in open_parens)
            single = any(re.search(r"\blane == 0\b", h) for h in open_blocks)
            found.append((src.count("\n", 0, i) + 1, voted or single))
        if ch == "(":
            open_parens.append(src[max(0, i - 32):i].rstrip())
        elif ch == ")":
            open_parens.pop()
        elif ch == "{":
            open_blocks.append(src[head:i])
        elif ch == "}":
            open_blocks.pop()
        if ch in "{};":
            head = i + 1
    assert not open_parens and not open_blocks
    return found


def test_the_scan_tells_the_forms_apart():
    one = "if (lane == 0) { while (x) { if (!mbar_wait(&b, p, a, e)) break; } }"
    vote = "void f() { ok = __all_sync(0xFFFFFFFFu, mbar_wait<P>(&b, p, a, e)); }"
    bare = "void f() { if (!mbar_wait<P>(&b, p, a, e)) break; }  // lane == 0"
    assert _waits(one) == [(1, True)] and _waits(vote) == [(1, True)]
    assert _waits(bare) == [(1, False)]


@pytest.mark.parametrize("name,least", [("gemm_fp8_block.cu", 4), ("gemm.cu", 6)])
def test_every_wait_is_one_lanes_or_voted(name, least):
    with open(os.path.join(CSRC, name)) as f:
        waits = _waits(f.read())
    assert len(waits) >= least
    assert not [line for line, ok in waits if not ok]
