"""Reference counts that fall short of what the tables hold are told of, by the update and by the
compaction, and counts that do not fall short never are."""
import random

import pytest
import torch

import speclib
from paged_kv_cache_251_gb300 import pa
from test_gpu_pages import check_update, run_compact, run_update, state

pytestmark = pytest.mark.gpu


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def update_flags(*args):
    err = word()
    got = check_update(*args, err=err)
    return got, err.item()


def test_update_kept_block_without_a_count():
    """Block 0 is held with a count of 0: it is handed out a second time, and that is told."""
    got, err = update_flags([[0, -1, -1]], [0, 0, 0], [4], None, [4], [8], 4)
    assert got[0] == [[0, 0, -1]] and err == pa.DEVERR_BAD_COUNT
    got, err = update_flags([[0, -1, -1]], [1, 0, 0], [4], None, [4], [8], 4)
    assert got[0] == [[0, 1, -1]] and err == 0
    # nothing grows: the row still holds a block that counts as free
    assert update_flags([[0, -1, -1]], [0, 0, 0], [4], None, [4], [4], 4)[1] == pa.DEVERR_BAD_COUNT
    # the row lets go of the block: the count falls below 0
    assert update_flags([[0, -1, -1]], [0, 0, 0], [4], None, [0], [0], 4)[1] == pa.DEVERR_BAD_COUNT


def test_update_two_rows_on_a_count_of_one():
    """Harmless while both keep the block; told as soon as one of them lets go."""
    tables, refs = [[2, 0, -1], [2, 1, -1]], [1, 1, 1, 0]
    assert update_flags(tables, refs, [8, 8], [0, -1], [8, 0], [8, 0], 4)[1] == pa.DEVERR_BAD_COUNT
    assert update_flags(tables, [1, 1, 2, 0], [8, 8], [0, -1], [8, 0], [8, 0], 4)[1] == 0


def test_update_copies_of_a_block_whose_count_is_short():
    """Three rows write behind one last block that counts one holder: no copy may take the last count."""
    tables, lens = [[0, -1], [0, -1], [0, -1]], [2, 2, 2]
    err = word()
    run_update(tables, [1, 0, 0, 0, 0], lens, None, lens, [3, 3, 3], 4, err=err)
    assert err.item() == pa.DEVERR_BAD_COUNT
    assert update_flags(tables, [3, 0, 0, 0, 0], lens, None, lens, [3, 3, 3], 4)[1] == 0
    assert update_flags(tables, [4, 0, 0, 0, 0], lens, None, lens, [3, 3, 3], 4)[1] == 0


def test_update_shortage_tells_of_counts():
    """Too few blocks: nothing changes, counts that are wrong are told of all the same."""
    got, err = update_flags([[0, 1, -1]], [1, 0, 1, 1], [8], None, [4], [12], 4)
    assert got[3][0] == 0 and err == pa.DEVERR_BAD_COUNT  # (block 1 falls to -1)
    got, err = update_flags([[0, 1, -1]], [1, 0, 1, 1], [8], None, [8], [12], 4)
    assert got[3][0] == 1 and err == pa.DEVERR_BAD_COUNT  # (block 1 suffices, twice)
    got, err = update_flags([[0, 1, -1, -1]], [1, 0, 1, 1], [8], None, [8], [16], 4)
    assert got[3][0] == 0 and err == pa.DEVERR_BAD_COUNT
    got, err = update_flags([[0, 1, -1, -1]], [1, 1, 1, 1], [8], None, [8], [16], 4)
    assert got[3][0] == 0 and err == 0


@pytest.mark.parametrize("rows,m,bs,nb", [(3, 5, 8, 0), (64, 40, 16, 0), (300, 20, 16, 70000), (1500, 3, 7, 0)])
def test_update_right_counts_are_never_flagged(rows, m, bs, nb):
    rng = random.Random(rows)
    for turn in range(3):
        tables, refs, lens = state(rng, rows, m, bs, True, max(nb, rng.choice([0, 10, 1000])))
        parents = [rng.choice([-1, i, i, rng.randrange(rows)]) for i in range(rows)]
        keep = [lens[p] if p >= 0 else 0 for p in parents]
        grow = [min(k + rng.choice([0, 1, bs]), m * bs) for k in keep]
        assert update_flags(tables, refs, lens, parents, keep, grow, bs)[1] == 0
        # one kept block's count at 0 is found wherever it is
        held = [(i, j) for i, p in enumerate(parents) for j in range(-(-keep[i] // bs)) if p >= 0]
        if held:
            i, j = rng.choice(held)
            b = tables[parents[i]][j]
            kept = sum(tables[p][:-(-keep[k] // bs)].count(b) for k, p in enumerate(parents) if p >= 0)
            had = sum(row[:-(-n // bs)].count(b) for row, n in zip(tables, lens))
            err = word()
            short = list(refs)
            short[b] = had - kept
            run_update(tables, short, lens, parents, keep, grow, bs, err=err)
            assert err.item() == pa.DEVERR_BAD_COUNT


@pytest.mark.parametrize("inplace", [False, True])
def test_compact_held_block_without_a_count(inplace):
    def flags(tables, refs, lens, moves=4):
        err = word()
        got = run_compact(tables, refs, lens, 4, moves, err=err, inplace=inplace)
        assert got == list(speclib.pages_compact(tables, refs, lens, 4, moves))
        return err.item()

    assert flags([[1, -1]], [0, 0, 1, 1], [4]) == pa.DEVERR_BAD_COUNT
    assert flags([[0, 2]], [0, 0, 1, 1], [8]) == pa.DEVERR_BAD_COUNT  # (block 2 moves onto block 0, which is held)
    assert flags([[0, 2]], [1, 0, 1, 1], [8]) == 0
    assert flags([[0, 2]], [1, 0, 1, 1], [8], moves=0) == 0
    assert flags([[0, 2]], [0, 0, 1, 1], [0]) == 0  # (behind lens nothing is held)
    rng = random.Random(7)
    for rows, m, bs in ((17, 9, 16), (900, 13, 16)):
        tables, refs, lens = state(rng, rows, m, bs, True, 900)
        err = word()
        run_compact(tables, refs, lens, bs, len(refs) // 2, err=err, inplace=inplace)
        assert err.item() == 0
        b = next(row[0] for row, n in zip(tables, lens) if n)
        refs[b] = 0
        run_compact(tables, refs, lens, bs, len(refs) // 2, err=err, inplace=inplace)
        assert err.item() == pa.DEVERR_BAD_COUNT
