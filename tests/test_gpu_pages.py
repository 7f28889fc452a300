"""Page tables on the device against the definition: rows kept, cut, forked, freed
and grown, copies of shared last blocks, shortage, compaction, copies; all exact."""
import random

import pytest
import torch

import speclib
from paged_kv_cache_251_gb300 import pa

pytestmark = pytest.mark.gpu


def cuda(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def run_update(tables, refs, lens, parents, keep, grow, bs, nb=None, err=None, stream=None):
    n, m = len(keep), len(tables[0])
    new = torch.full((n, m), -9, dtype=torch.int32, device="cuda")
    new_refs = torch.full((len(refs),), -9, dtype=torch.int32, device="cuda")
    pairs = torch.full((n, 2), -9, dtype=torch.int64, device="cuda")
    status = torch.full((4,), -9, dtype=torch.int32, device="cuda")
    pa.pa_pages_update(new, new_refs, pairs, status, cuda(tables), cuda(refs), cuda(lens), cuda(keep), cuda(grow), bs,
                       parents=None if parents is None else cuda(parents), err_word=err, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().tolist() for x in (new, new_refs, pairs, status)]


def check_update(tables, refs, lens, parents, keep, grow, bs, err=None):
    got = run_update(tables, refs, lens, parents, keep, grow, bs, err=err)
    want = speclib.pages_update(tables, refs, lens, parents, keep, grow, bs)
    if want[0] is None:
        assert got[2:] == list(want[2:])
        assert all(x == -9 for row in got[0] for x in row) and all(x == -9 for x in got[1])
    else:
        assert got == list(want)
    return got


def state(rng, rows, m, bs, share, spare):
    """Random tables with a common prefix for some neighbours, and their counts."""
    lens = [rng.choice([0, 1, bs, rng.randint(0, m * bs), rng.randint(0, m * bs)]) for _ in range(rows)]
    need = rows * m + spare
    order = list(range(need))
    rng.shuffle(order)
    tables, refs = [], [0] * need
    it = iter(order)
    for r in range(rows):
        n = -(-lens[r] // bs)
        row = []
        if share and r and rng.random() < 0.6:
            other = tables[r - 1]
            have = -(-lens[r - 1] // bs)
            row = other[:rng.randint(0, min(n, have))]
        row = row + [next(it) for _ in range(n - len(row))]
        for b in row:
            refs[b] += 1
        tables.append(row + [-1] * (m - n))
    # keep the pool small: what is free, and some of it held elsewhere
    for b in order:
        if refs[b] == 0 and rng.random() < 0.1:
            refs[b] = rng.randint(1, 3)
    return tables, refs, lens


@pytest.mark.parametrize("rows,m,bs", [(1, 1, 16), (3, 5, 8), (17, 9, 16), (64, 40, 32), (300, 20, 16), (5, 2100, 16),
                                       (1500, 3, 7)])
@pytest.mark.parametrize("share", [False, True])
def test_update_random(rows, m, bs, share):
    rng = random.Random(rows * 10 + share)
    for turn in range(4):
        tables, refs, lens = state(rng, rows, m, bs, share, rng.choice([0, 10, 1000]))
        n = rows if turn < 2 else rng.randint(1, 2 * rows)
        parents = [rng.choice([-1, i % rows, rng.randrange(rows), rng.randrange(rows)]) for i in range(n)]
        if turn == 0:
            parents = None
        keep = [rng.randint(-1, m * bs + 3) for _ in range(n)]
        grow = [max(0, k) + rng.choice([0, 1, bs, 3 * bs]) for k in keep]
        grow = [min(g, m * bs) for g in grow]
        check_update(tables, refs, lens, parents, keep, grow, bs)


def test_update_beam_search_loops():
    """Forks of forks: last blocks shared by several, the first writer stays only where all write."""
    rng = random.Random(5)
    bs, m, rows, nb = 4, 12, 8, 120
    tables, refs, lens = [[-1] * m for _ in range(rows)], [0] * nb, [0] * rows
    for step in range(40):
        parents = [rng.randrange(rows) for _ in range(rows)]
        keep = [lens[p] for p in parents]
        grow = [min(k + rng.choice([0, 1, 1, 3]), m * bs) for k in keep]
        if max(grow) > m * bs - 4:
            keep = [0] * rows
            grow = [rng.randint(0, 5) for _ in range(rows)]
        tables, refs, pairs, status = check_update(tables, refs, lens, parents, keep, grow, bs)
        assert status[0] == 1
        lens = grow
        held = [b for row, n in zip(tables, lens) for b in row[:-(-n // bs)]]
        assert all(refs[b] == held.count(b) for b in range(nb))


def test_update_shortage_changes_nothing():
    tables, refs, lens = [[0, 1, -1, -1], [2, -1, -1, -1]], [1, 1, 1, 0, 5], [8, 3]
    got = check_update(tables, refs, lens, None, [8, 3], [13, 4], 4)
    assert got[3] == [0, 2, 1, 0]
    got = check_update(tables, refs, lens, None, [8, 3], [12, 4], 4)
    assert got[3] == [1, 1, 0, 0]
    # what the rows let go in the same call counts as free
    got = check_update(tables, refs, lens, [0, -1], [0, 0], [16, 0], 4)
    assert got[3] == [1, 4, 0, 0] and got[0][0] == [0, 1, 2, 3]


def test_update_blocks_held_elsewhere_are_copied():
    """A prompt cache's reference on the last block: its rows stay as they are."""
    got = check_update([[3, 1, -1]], [0, 2, 0, 1], [6], None, [6], [7], 4)
    assert got[2] == [[1, 0]] and got[1] == [1, 1, 0, 1]
    got = check_update([[3, 1, -1]], [0, 1, 0, 1], [6], None, [6], [7], 4)
    assert got[2] == [[-1, -1]]
    got = check_update([[3, 1, -1]], [0, 2, 0, 1], [6], None, [6], [6], 4)  # nothing is written
    assert got[2] == [[-1, -1]]


def test_update_flags_bad_contents_in_a_shortage():
    """Nothing changes, but the entry outside the pool that a row would have kept is told of."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = check_update([[9, 1, -1]], [0, 1, 1, 1], [8], [0], [8], [12], 4, err=err)
    assert got[3][0] == 1 and err.item() == pa.DEVERR_BAD_BLOCK  # (block 0 is free: it suffices)
    err.zero_()
    got = check_update([[9, 1, -1]], [1, 1, 1, 1], [8], [0], [8], [12], 4, err=err)
    assert got[3] == [0, 1, 0, 0] and err.item() == pa.DEVERR_BAD_BLOCK
    err.zero_()
    got = check_update([[3, 1, -1]], [1, 1, 1, 1], [8], [0], [8], [12], 4, err=err)
    assert got[3] == [0, 1, 0, 0] and err.item() == 0


def test_update_bad_contents():
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_update([[9, 1, -1], [2, -4, -1]], [0, 1, 1, 0], [6, 5], [0, 1], [6, 5], [6, 5], 4, err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK
    err.zero_()
    check_update([[0, 1, -1]], [1, 1, 0, 0], [99], [7], [1], [99], 4, err=err)
    assert err.item() == pa.DEVERR_BAD_INDEX | pa.DEVERR_BAD_LEN | pa.DEVERR_BAD_BLOCK  # (lens 99 reaches the -1)
    err.zero_()
    run_update([[0, 1, -1]], [1, 0, 0, 0], [8], [-1], [0], [0], 4, err=err)
    assert err.item() == pa.DEVERR_BAD_COUNT


def test_update_in_place_counts_and_no_rows():
    refs = cuda([1, 1, 0, 0])
    new, pairs, status = (torch.empty((1, 3), dtype=torch.int32, device="cuda"),
                          torch.empty((1, 2), dtype=torch.int64, device="cuda"), cuda([0, 0, 0, 0]))
    pa.pa_pages_update(new, refs, pairs, status, cuda([[1, 0, -1]]), refs, cuda([8]), cuda([8]), cuda([9]), 4)
    assert refs.tolist() == [1, 1, 1, 0] and new.tolist() == [[1, 0, 2]] and status.tolist() == [1, 1, 1, 0]
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    pa.pa_pages_update(none, refs, torch.empty((0, 2), dtype=torch.int64, device="cuda"), status, new, refs, cuda([9]),
                       empty, empty, 4, parents=empty)
    assert refs.tolist() == [0, 0, 0, 0] and status.tolist() == [1, 0, 4, 0]


def run_compact(tables, refs, lens, bs, max_moves, err=None, inplace=False):
    t, r = cuda(tables), cuda(refs)
    new, new_refs = (t, r) if inplace else (torch.full_like(t, -9), torch.full_like(r, -9))
    remap = torch.full_like(r, -9)
    pairs = torch.full((max_moves, 2), -9, dtype=torch.int64, device="cuda")
    status = cuda([0] * 4)
    pa.pa_pages_compact(new, new_refs, remap, pairs, status, t, r, cuda(lens), bs, err_word=err)
    torch.cuda.synchronize()
    return [x.cpu().tolist() for x in (new, new_refs, remap, pairs, status)]


@pytest.mark.parametrize("rows,m,bs", [(1, 1, 16), (3, 5, 8), (17, 9, 16), (64, 40, 32), (5, 2100, 16), (900, 13, 16)])
def test_compact_random(rows, m, bs):
    rng = random.Random(rows)
    for turn in range(3):
        tables, refs, lens = state(rng, rows, m, bs, True, rng.choice([0, 10, 9000]))
        for moves in (len(refs) // 2, 3, 0):
            want = speclib.pages_compact(tables, refs, lens, bs, moves)
            assert run_compact(tables, refs, lens, bs, moves, inplace=turn == 1) == list(want)


def test_compact_ends():
    for refs in ([0] * 7, [1] * 7, [0, 0, 0, 0, 0, 0, 2], [3, 0, 0, 0, 0, 0, 0], [1]):
        want = speclib.pages_compact([[-1, -1]], refs, [0], 4, 5)
        assert run_compact([[-1, -1]], refs, [0], 4, 5) == list(want)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_compact([[5, 77]], [0, 0, 0, 0, -1, 1], [900], 4, 2, err=err)
    assert got == list(speclib.pages_compact([[5, 77]], [0, 0, 0, 0, -1, 1], [900], 4, 2))
    assert err.item() == pa.DEVERR_BAD_BLOCK | pa.DEVERR_BAD_LEN | pa.DEVERR_BAD_COUNT


@pytest.mark.parametrize("shapes", [[((2, 16, 64), torch.float16)], [((8, 32, 128), torch.int8), ((8,), torch.float32)],
                                    [((1,), torch.float32), ((3, 5), torch.float32), ((1, 8, 64), torch.bfloat16)],
                                    [((40, 16, 128), torch.float32)] * 8])
@pytest.mark.parametrize("n", [0, 1, 100, 3000])
def test_copy(shapes, n):
    gen = torch.Generator().manual_seed(n)
    nb = 2 * n + 3 if shapes[0][0][0] < 40 else min(2 * n + 3, 203)
    n = min(n, (nb - 3) // 2)
    order = torch.randperm(nb, generator=gen)
    pairs = torch.stack([order[:n], order[n:2 * n]], 1).contiguous()
    if n > 2:
        pairs[::3] = torch.tensor([-1, -1])
    pools = [torch.randn((nb,) + s, generator=gen).mul(50).to(t).cuda() for s, t in shapes]
    want = [p.clone() for p in pools]
    good = pairs[pairs[:, 0] >= 0].cuda()
    for w in want:
        w[good[:, 1]] = w[good[:, 0]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_copy_pages(pairs.cuda(), pools, err_word=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copy_flags_pairs_outside_the_pool():
    pool = torch.arange(40, dtype=torch.float32, device="cuda").view(10, 4).contiguous()
    want = pool.clone()
    want[4] = want[2]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_copy_pages(cuda([[10, 1], [2, 4], [3, -1], [3, 10], [-1, 5]], torch.int64), [pool], err_word=err)
    assert torch.equal(pool, want) and err.item() == pa.DEVERR_BAD_PAIR


def test_update_in_a_graph_with_its_copies():
    """A captured step that ends where it began: replayed, it walks two tables in turn."""
    bs, m, nb = 4, 8, 40
    refs, lens = cuda([1, 1, 1] + [0] * (nb - 3)), cuda([10, 10])
    a = cuda([[0, 1, 2] + [-1] * 5, [-1] * 8])
    b = torch.empty_like(a)
    pool = torch.randn(nb, 16, device="cuda")
    before = pool.clone()
    pairs, status = torch.empty((2, 2), dtype=torch.int64, device="cuda"), cuda([0] * 4)
    new_refs = torch.empty_like(refs)
    args = dict(parents=cuda([0, 0]), workspace=pa.pages_workspace_for(a, refs))
    lens0 = cuda([10, 0])

    def step():
        pa.pa_pages_update(b, new_refs, pairs, status, a, refs, lens0, lens, cuda_grow, bs, **args)
        pa.pa_copy_pages(pairs, [pool])

    cuda_grow = cuda([11, 11])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    b.fill_(-3)
    args["workspace"].fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    want = speclib.pages_update(a.tolist(), refs.tolist(), [10, 0], [0, 0], [10, 10], [11, 11], bs)
    assert [b.tolist(), new_refs.tolist(), pairs.tolist(), status.tolist()] == list(want)
    assert torch.equal(pool[3], before[2]) and want[2] == [[-1, -1], [2, 3]]
