"""A model of who touches the output accumulators of the tensor-core tree
attention (csrc/pa_tree_tc.cuh) with at most 128 rows a kv head, over every
interleaving, on the CPU.

Two warpgroups share an item's rows, each with its own accumulator O in tensor
memory.  In an item's epilogue both read both; in the first tile of an item a
warpgroup may write its own (a drafted token with a non-finite V row), and the
P V warp's products write both.  Whoever writes O for an item has to wait for
the epilogues of the item before (the barrier `ofree`).  Whether the kernel's
two writers do is read from its source."""
import re
from pathlib import Path

import pytest

import paged_kv_cache_251_gb300

SOURCE = (Path(paged_kv_cache_251_gb300.__file__).parent / "csrc" / "pa_tree_tc.cuh").read_text()


def waits_before(begin, end):
    """Whether `ofree` is waited for between two places of the source."""
    a = SOURCE.index(begin)
    return "&M->ofree" in SOURCE[a:SOURCE.index(end, a)]


def explore(items, draft_waits, pv_waits):
    """Every interleaving of three actors over `items`, a list of flags: the item
    has a non-finite draft in its first tile.  Raises where O is written before
    both epilogues of the item before have read it, or where all are stuck."""
    n = len(items)

    def warpgroup(w):
        for k, bad in enumerate(items):
            if bad:
                if draft_waits and k:
                    yield ("wait", "ofree", k)
                yield ("write", k)
            yield ("arrive", "pfull", w)
            yield ("wait", "odone", k + 1)
            yield ("arrive", "xbar", 0)
            yield ("wait", "xbar", k + 1)
            yield ("read", k)
            yield ("arrive", "ofree", 0)

    def pv():
        for k in range(n):
            yield ("wait", "pfull0", k + 1)
            if pv_waits and k:
                yield ("wait", "ofree", k)
            yield ("write", k)
            yield ("wait", "pfull1", k + 1)
            yield ("write", k)
            yield ("arrive", "odone", 0)

    programs = [list(warpgroup(0)), list(warpgroup(1)), list(pv())]
    count = {"ofree": 2, "xbar": 2}     # arrivals of a phase (a warpgroup as one)
    seen, todo = set(), [((0, 0, 0), (), (0, 0))]

    def phases(arrived, name):
        return dict(arrived).get(name, 0) // count.get(name, 1)

    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        at, arrived, read = state
        moved = False
        for a, program in enumerate(programs):
            if at[a] == len(program):
                continue
            op, *arg = program[at[a]]
            if op == "wait" and phases(arrived, arg[0]) < arg[1]:
                continue
            moved = True
            now, got = dict(arrived), list(read)
            if op == "arrive":
                name = f"pfull{arg[1]}" if arg[0] == "pfull" else arg[0]
                now[name] = now.get(name, 0) + 1
            elif op == "write":
                assert min(read) >= arg[0], f"O of item {arg[0]} written while the epilogue before still reads it"
            elif op == "read":
                got[a] += 1
            todo.append((tuple(x + (i == a) for i, x in enumerate(at)), tuple(sorted(now.items())), tuple(got)))
        assert moved or all(x == len(p) for x, p in zip(at, programs)), f"stuck at {at}"


ITEMS = [[False, True], [True, True], [True, False, True], [True, True, True]]


@pytest.mark.parametrize("items", ITEMS)
def test_accumulators_are_written_after_the_epilogue_before(items):
    explore(items, waits_before("if (poisoned) {", "tmem_st16(o_addr"),
            waits_before("inline bool tc_pv_warp(", "tc_mma_ts(lead"))


@pytest.mark.parametrize("draft_waits,pv_waits", [(False, True), (True, False)])
def test_the_model_sees_a_missing_wait(draft_waits, pv_waits):
    with pytest.raises(AssertionError, match="written while"):
        explore([False, not draft_waits], draft_waits, pv_waits)


def test_words_of_the_source():
    """What the model takes from the source is there once."""
    assert SOURCE.count("if (poisoned) {") == 1
    assert len(re.findall(r"mbar_arrive\(&M->ofree\)", SOURCE)) == 1
    assert "mbar_init(&M->ofree, 8);" in SOURCE


def test_arrivals_for_a_warp_come_after_its_lanes():
    """In the softmax one lane arrives for its warp, whose lanes have all written
    something (weights, zeroed V rows, an accumulator): each such arrival follows a
    __syncwarp() directly, and nothing that diverges lies between."""
    body = SOURCE[SOURCE.index("inline bool tc_softmax("):SOURCE.index("pa_tree_tc_kernel(const TreeParams p")]
    lines = [x.split("//")[0].strip() for x in body.splitlines()]
    lines = [x for x in lines if x]
    at = [i for i, x in enumerate(lines) if x.startswith("mbar_arrive(")]
    assert len(at) >= 6
    for i in at:
        assert lines[i - 1] == "if (lane == 0)" and lines[i - 2] == "__syncwarp();", lines[i - 3:i + 1]
