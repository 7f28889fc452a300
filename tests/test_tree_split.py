"""The even split of tree attention, on the CPU: the tiles of all (sequence, kv
head, row tile) pairs, each pair counted with a fixed cost before its tiles, cut
into equal spans.  A model of the device's rule (csrc/pa_tree_tc.cuh: tc_find,
TcWalk, the merge's records) is held to what the kernels rely on."""
import random
import re
from pathlib import Path

import pytest

import paged_kv_cache_251_gb300

SOURCE = Path(paged_kv_cache_251_gb300.__file__).parent / "csrc" / "pa_tree_tc.cuh"
COST = int(re.search(r"constexpr int kTcPairCost = (\d+);", SOURCE.read_text()).group(1))


def split(tiles, pairs_per_seq, ctas):
    """Every CTA's items (pair, first tile, end, slot) and its merge records: by
    slot, (pair, first CTA, parts) or None."""
    pairs = [t for t in tiles for _ in range(pairs_per_seq)]
    starts, total = [], 0
    for t in pairs:
        starts.append(total)
        total += t + COST
    spans = min(ctas, max(total, 1))
    items, records = [], []
    for c in range(ctas):
        mine, record = [], [None, None]
        if c < spans:
            u0, u1 = total * c // spans, total * (c + 1) // spans
            for i, (t, start) in enumerate(zip(pairs, starts)):
                lo, hi = (max(0, min(t, u - start - COST)) for u in (u0, u1))
                if start >= u1 or not (hi > lo or (t == 0 and start >= u0)):
                    continue
                slot = -1 if hi - lo == t else (0 if lo > 0 else 1)
                if slot >= 0:
                    first = ((start + COST + 1) * spans - 1) // total
                    record[slot] = (i, first, ((start + COST + t) * spans - 1) // total - first + 1)
                mine.append((i, lo, hi, slot))
        items.append(mine)
        records.append(record)
    return pairs, items, records


@pytest.mark.parametrize("seed", range(6))
def test_even_split(seed):
    r = random.Random(seed)
    for _ in range(400):
        tiles = [r.choice([0, 1, 1, 2, 3, r.randint(0, 40)]) for _ in range(r.randint(1, 20))]
        pairs, items, records = split(tiles, r.choice([1, 2, 3, 8]), r.choice([1, 2, 5, 48, 152]))
        parts = {}
        for c, mine in enumerate(items):
            slots = [slot for *_, slot in mine if slot >= 0]
            assert len(slots) == len(set(slots))           # at most two partials a CTA, in their own slots
            for i, lo, hi, slot in mine:
                parts.setdefault(i, []).append((lo, hi, c, slot))
        cut = set()
        for i, t in enumerate(pairs):
            segs = sorted(parts[i])                        # every pair is somewhere, an empty one once
            assert segs[0][0] == 0 and segs[-1][1] == t
            assert all(a[1] == b[0] for a, b in zip(segs, segs[1:]))
            assert len(segs) == 1 or t > 1
            if len(segs) > 1:
                cut.add(i)
        assert {rec[0] for both in records for rec in both if rec} == cut
        for c, both in enumerate(records):
            for slot, rec in enumerate(both):
                if rec:                                    # partial 1 of the first CTA, partial 0 of those after it
                    i, first, n = rec
                    want = [(first, 1)] + [(first + q, 0) for q in range(1, n)]
                    assert [(cc, sl) for _, _, cc, sl in sorted(parts[i])] == want and (c, slot) in want
        assert sum(rec is not None for both in records for rec in both) == sum(len(parts[i]) for i in cut)


def test_spans_are_even():
    """With contexts far longer than the cost, no CTA has more than its share of
    tiles and one."""
    for ctas in (7, 152):
        _, items, _ = split([900, 1500, 2, 3000], 8, ctas)
        work = [sum(hi - lo + COST * (lo == 0) for _, lo, hi, _ in mine) for mine in items]
        share = 8 * (900 + 1500 + 2 + 3000 + 4 * COST) / ctas
        assert max(work) <= share + COST + 1 and min(work) >= share - COST - 1
