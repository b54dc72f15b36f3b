"""Registers that the warps of the prompts' attention kernel hand to one another.

The kernel's CTA owns what it was launched with (512 threads x 128).  Its copy
and MMA warps give registers up, its softmax warps take them, and before the
common tail both sides go back to the launch count.  A warp that asks for more
than is free waits, and no time limit covers that wait, so the order of the
changes has to make sure that it ends.  Here the order is read from the source,
and every interleaving of the sixteen warps is walked through on the host.
"""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "long_context_decode_basiskv_b200", "csrc", "dense_attn_tc.cu")
LAUNCH, WARPS = 128, 16


def branches():
    """The register changes and barriers of the two branches, in source order: ("set", text) and ("bar", id,
    threads) with ids and counts as they are written.  The end of the kernel's branches is ("end",)."""
    s = open(SOURCE).read()
    start = s.index("  if (warp < 8) {\n")
    middle = s.index("\n  } else {\n", start)
    end = s.index("  if (!ok) set_err(p.err, BASISKV_DEVERR_TIMEOUT);", middle)
    step = re.compile(r'setmaxnreg\.(?:inc|dec)\.sync\.aligned\.u32 %0;" ::"n"\((.+)\)\);|dt_bar<(\d+), (\w+)>\(\);|'
                      r'bar\.sync (\w+), (\w+);')
    out = []
    for part in (s[start:middle], s[middle:end]):
        ops = []
        for x in step.finditer(part):
            if x.group(1):
                ops.append(("set", x.group(1)))
            else:
                ops.append(("bar", x.group(2) or x.group(4), x.group(3) or x.group(5)))
        out.append(ops + [("end",)])
    return out


def programs(softmax_regs, one_row_tile):
    """What each of the sixteen warps runs, with numbers in place of the source's names."""
    count = {"dt_regs<RMAX>()": softmax_regs, "256 - dt_regs<RMAX>()": 256 - softmax_regs, "128": LAUNCH}
    soft, rest = branches()
    # a barrier that only CTAs of one row tile pass: the two warpgroups join their results
    assert [op for op in soft if op[0] == "bar" and op[1] == "1"] == [("bar", "1", "256")] * 2
    joins = soft.index(("bar", "1", "256"))
    if not one_row_tile:
        soft = soft[:joins] + soft[joins + 1:]
    progs = []
    for w in range(WARPS):
        prog = []
        for op in (soft if w < 8 else rest):
            if op[0] == "set":
                prog.append(("set", count[op[1]]))
            elif op[0] == "bar":
                threads = 32 * WARPS if op[2] == "kDtThreads" else int(op[2])
                prog.append(("bar", int(op[1]), threads // 32))
        progs.append(prog + [("bar", 0, WARPS)])
    return progs


def stuck(progs):
    """A reachable state in which some warp has not finished and none can go on, or None.  Warps with equal
    programs are interchangeable, so a state is how many of each kind stand where."""
    kinds = sorted(set(map(tuple, progs)))
    many = [sum(tuple(p) == k for p in progs) for k in kinds]
    first = tuple(tuple([n] + [0] * len(k)) for k, n in zip(kinds, many))

    def regs_of(k, pc):
        held = LAUNCH
        for op in k[:pc]:
            if op[0] == "set":
                held = op[1]
        return held
    held = [[regs_of(k, pc) for pc in range(len(k) + 1)] for k in kinds]
    seen, todo = {first}, [first]
    while todo:
        at = todo.pop()
        free = LAUNCH * WARPS - sum(n * held[x][pc] for x, row in enumerate(at) for pc, n in enumerate(row))
        assert free >= 0
        moves = []
        waiting = {}
        for x, row in enumerate(at):
            for pc, n in enumerate(row[:-1]):
                if not n:
                    continue
                op = kinds[x][pc]
                if op[0] == "set":
                    if op[1] - held[x][pc] <= free:
                        moves.append([(x, pc, 1)])
                else:
                    waiting.setdefault(op[1:], []).append((x, pc, n))
        for (ident, warps), who in waiting.items():
            if sum(n for _, _, n in who) == warps:
                moves.append(who)
        if not moves and any(sum(row[:-1]) for row in at):
            return at
        for move in moves:
            new = [list(row) for row in at]
            for x, pc, n in move:
                new[x][pc] -= n
                new[x][pc + 1] += n
            new = tuple(map(tuple, new))
            if new not in seen:
                seen.add(new)
                todo.append(new)
    return None


@pytest.mark.parametrize("softmax_regs", [208, 216, 224])
@pytest.mark.parametrize("one_row_tile", [False, True])
def test_every_order_of_the_warps_ends(softmax_regs, one_row_tile):
    progs = programs(softmax_regs, one_row_tile)
    assert [op for op in progs[0] if op[0] == "set"] == [("set", softmax_regs), ("set", LAUNCH)]
    assert [op for op in progs[15] if op[0] == "set"] == [("set", 256 - softmax_regs), ("set", LAUNCH)]
    assert stuck(progs) is None


def test_the_walk_finds_a_tail_that_takes_registers_too_early():
    """Both sides restoring their count with nothing between them: an idle warp's request can come first."""
    early = [[("set", 208), ("set", LAUNCH), ("bar", 0, WARPS)]] * 8 + [[("set", 48), ("set", LAUNCH), ("bar", 0, WARPS)]] * 8
    assert stuck(early) is not None


@pytest.mark.parametrize("softmax_regs", [208, 224])
@pytest.mark.parametrize("one_row_tile", [False, True])
def test_a_warpgroup_meets_between_two_changes(softmax_regs, one_row_tile):
    """All warps of a warpgroup synchronise between two setmaxnreg instructions."""
    progs = programs(softmax_regs, one_row_tile)
    for group in range(4):
        for w in range(4 * group, 4 * group + 4):
            changes = [x for x, op in enumerate(progs[w]) if op[0] == "set"]
            for a, b in zip(changes, changes[1:]):
                assert any(op[0] == "bar" and op[2] >= 4 for op in progs[w][a + 1:b]), (w, progs[w])
