"""What the tree attention's softmax warps hand each other between pieces, as a model of the kernel's order of events:
with the buffers that the source has, no warp, however late, reads what a later piece has overwritten; with fewer one does.

The model: twelve warps, three groups by four quarters of the rows; a piece of some blocks, block k the (k % 3)rd group's.
An event waits for others and counts, writes a slot or reads it.  No event chooses, so holding one warp back before a
read and letting all others go as far as they can shows everything that may happen before that read."""
import itertools
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GROUPS, QUARTERS, BUFS = 3, 4, 6
WARPS = [(g, q) for g in range(GROUPS) for q in range(QUARTERS)]


def programs(sizes):
    """Each warp's events: (kind, what), of the pieces of `sizes` blocks."""
    first = [0] + list(itertools.accumulate(sizes))
    out = {}
    for g, q in WARPS:
        ev = [("write", "scales", 0), ("arrive", "qready", 0)]
        for p, n in enumerate(sizes):
            if p + 1 < len(sizes):
                ev += [("write", "scales", p + 1), ("arrive", "qready", p + 1)]
            ev += [("wait", "qready", p), ("read", "scales", p)]
            for k in range(first[p], first[p] + n):
                if k % GROUPS == g:
                    ev += [("wait", "token", (k - 1, q)), ("wait", "s", k), ("write", "mark", p), ("arrive", "token", (k, q)),
                           ("arrive", "pfull", k)]
            ev += [("wait", "pv", first[p + 1] - 1), ("read", "mark", p), ("write", "sums", p), ("arrive", "lfull", (p, q)),
                   ("wait", "lfull", (p, q)), ("read", "sums", p), ("arrive", "ofree", p)]
        out[g, q] = ev
    return out


def run(sizes, slots, held, at):
    """All warps as far as they go, `held` stopped before its event `at`; the newest piece in each slot."""
    first = [0] + list(itertools.accumulate(sizes))
    piece_of = [p for p, n in enumerate(sizes) for _ in range(n)]
    ev, pc = programs(sizes), dict.fromkeys(WARPS, 0)
    count, newest = {}, {}
    s = pv = 0  # blocks whose S and PV are done

    def reached(what, x):
        if what == "token":
            return x[0] < 0 or count.get((what, x), 0) >= 1
        if what == "s":
            return s > x
        if what == "pv":
            return pv > x
        return count.get((what, x), 0) >= {"qready": 12, "lfull": GROUPS}[what]

    moved = True
    while moved:
        moved = False
        while s < first[-1] and count.get(("qready", piece_of[s]), 0) == 12 and s - BUFS < pv:
            s, moved = s + 1, True
        while (pv < s and count.get(("pfull", pv), 0) == QUARTERS and
               (piece_of[pv] == 0 or pv != first[piece_of[pv]] or count.get(("ofree", piece_of[pv] - 1), 0) == 12)):
            pv, moved = pv + 1, True
        for w in WARPS:
            while pc[w] < len(ev[w]) and not (w == held and pc[w] == at):
                kind, what, x = ev[w][pc[w]]
                if kind == "wait" and not reached(what, x):
                    break
                if kind == "arrive":
                    count[what, x] = count.get((what, x), 0) + 1
                if kind == "write":
                    key = (what, x % slots[what])
                    newest[key] = max(newest.get(key, x), x)
                pc[w], moved = pc[w] + 1, True
    return newest, all(pc[w] == len(ev[w]) for w in WARPS if w != held), held is None or pc[held] == at


def overwritten(sizes, slots):
    """The kinds of slots that some late warp may read too late."""
    found = set()
    for w, events in programs(sizes).items():
        for at, (kind, what, x) in enumerate(events):
            if kind != "read":
                continue
            newest, _, there = run(sizes, slots, w, at)
            assert there  # the others do not wait for good before it gets there
            if newest[what, x % slots[what]] > x:
                found.add(what)
    return found


def source():
    text = open(os.path.join(ROOT, "fp8_quantized_paged_gb300", "csrc", "kvq_tree.cuh")).read()
    value = lambda name: int(re.search(rf"constexpr int {name} = (\d+);", text).group(1))  # noqa: E731
    assert value("kBufs") == BUFS
    assert "ls_s[(n % kScaleBufs) * kRows + at]" in text and "ls_s[(piece % kScaleBufs) * kRows + r]" in text
    assert "vnan[piece % kNanMarks] = 1u + piece" in text and "vnan[piece % kNanMarks] == 1u + piece" in text
    assert "float2* sums = l_s + (piece & 1) * kGroups * kRows" in text
    return {"scales": value("kScaleBufs"), "mark": value("kNanMarks"), "sums": 2}


@pytest.mark.parametrize("sizes", [s + (2, 1) for s in itertools.product((1, 2, 5), repeat=3)] + [(7, 8, 2, 9), (1,) * 9])
def test_no_warp_reads_too_late(sizes):
    assert overwritten(sizes, source()) == set()


def test_fewer_slots_would_not_do():
    sizes, have = (2, 2, 2, 2, 1), source()
    for what in ("scales", "mark"):
        assert overwritten(sizes, dict(have, **{what: have[what] - 1})) == {what}


def test_the_model_runs_to_its_end():
    assert run((1, 2, 3, 9, 1), source(), None, None)[1]
