"""Fresh blocks for several sequences at once: the destinations of one eviction."""
import pytest
import torch

from paged_kv_cache_251_gb300 import workloads as wl

INV, NOBLK = 1, 5


def manager(num_blocks, bs, lens, max_blocks=8):
    from paged_kv_cache_251_gb300.blocks import BlockManager
    bm = BlockManager(num_blocks, bs, len(lens) + 1, max_blocks)
    for s, n in enumerate(lens):
        bm.add_sequence(s)
        bm.extend(s, n)
    return bm


def used(tables):
    return set(tables[tables >= 0].tolist())


def state(bm, num_blocks):
    tables, lens = bm.tables()
    return tables.tolist(), lens.tolist(), [bm.refcount(b) for b in range(num_blocks)], bm.num_free()


def test_no_destination_is_a_source():
    """Six blocks of three sequences, and a free list that covers all destinations
    exactly: none of them is a block that the sequences held."""
    bm = manager(9, 8, [16, 16, 16])
    before, _ = bm.tables()
    bm.renew_batch([0, 1, 2], [8, 3, 5])
    after, lens = bm.tables()
    assert lens.tolist() == [8, 3, 5, 0] and len(used(after)) == 3
    assert not used(before) & used(after)
    assert bm.num_free() == 6 and sorted(bm.refcount(b) for b in range(9)) == [0] * 6 + [1] * 3


def test_a_free_list_for_some_but_not_all_is_refused():
    """One destination fits, all do not: refused with nothing changed (one after the
    other would give the first sequence's old blocks to the others)."""
    from paged_kv_cache_251_gb300 import pa
    bm = manager(8, 8, [16, 16, 16])
    want = state(bm, 8)
    with pytest.raises(pa.PagedAttentionError) as e:
        bm.renew_batch([0, 1, 2], [8, 8, 8])
    assert e.value.status == NOBLK and state(bm, 8) == want
    one_by_one = manager(8, 8, [16, 16, 16])
    before, _ = one_by_one.tables()
    for s in range(3):
        one_by_one.renew(s, 8)
    assert used(before) & used(one_by_one.tables()[0])     # why: a source is a destination


@pytest.mark.parametrize("seqs,lens", [([0, 0], [8, 8]), ([0, 3], [8, 8]), ([0, 9], [8, 8]), ([0, -1], [8, 8]),
                                       ([0, 1], [8, -1]), ([0, 1], [8, 65]), ([0, 2], [8, 8])])
def test_refusals_change_nothing(seqs, lens):
    """A sequence twice, one that is not there, a negative or too long length, a window ring."""
    from paged_kv_cache_251_gb300 import pa
    bm = manager(40, 8, [16, 16])
    bm.add_sequence(2, ring_blocks=2)
    want = state(bm, 40)
    with pytest.raises(pa.PagedAttentionError) as e:
        bm.renew_batch(seqs, lens)
    assert e.value.status == INV and state(bm, 40) == want


def test_shared_blocks_keep_their_other_owner():
    bm = manager(12, 8, [16, 16])
    bm.fork(0, 2)
    before, _ = bm.tables()
    bm.renew_batch([0, 1], [16, 0])
    after, lens = bm.tables()
    assert lens.tolist() == [16, 0, 16] and after[2].tolist() == before[0].tolist()
    assert not used(after[0]) & used(before)
    assert [bm.refcount(b) for b in before[0, :2].tolist()] == [1, 1]
    bm.renew_batch([], [])
    with pytest.raises(ValueError):
        bm.renew_batch([0, 1], [8])


@pytest.mark.gpu
def test_one_eviction_of_many_sequences_with_a_short_free_list():
    """Twelve sequences evicted by one call into blocks that just suffice: every row
    is the kept one's."""
    from paged_kv_cache_251_gb300 import pa
    bs, hkv, d, n_seqs, budget = 8, 2, 64, 12, 20
    lens = [40 + 2 * s for s in range(n_seqs)]
    held, more = sum((n + bs - 1) // bs for n in lens), n_seqs * ((budget + bs - 1) // bs)
    bm = manager(held + more, bs, lens)
    assert bm.num_free() == more
    k = wl.normal_tensor(51, 4, (held + more, hkv, bs, d), dtype=torch.bfloat16).cuda()
    v = wl.normal_tensor(51, 5, (held + more, hkv, bs, d), dtype=torch.bfloat16).cuda()
    k0, v0 = k.clone(), v.clone()
    tables, lens_t = bm.tables()
    tables, lens_t = tables[:n_seqs].contiguous(), lens_t[:n_seqs].contiguous().cuda()
    scores = torch.rand((n_seqs, hkv, tables.shape[1] * bs), device="cuda")
    keep = torch.empty((n_seqs, hkv, budget), dtype=torch.int32, device="cuda")
    new = torch.empty(n_seqs, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new, scores, scores, lens_t, budget=budget, recent=4, err_word=err)
    bm.renew_batch(range(n_seqs), [budget] * n_seqs)
    dst = bm.tables()[0][:n_seqs].contiguous()
    pa.pa_compact_kv(k, v, keep, new, tables.cuda(), dst_block_tables=dst.cuda(), err_word=err)
    assert err.item() == 0 and bm.num_free() == held
    for s in range(n_seqs):
        for h in range(hkv):
            for i, j in enumerate(keep[s, h].tolist()):
                a, b = int(tables[s, j // bs]), int(dst[s, i // bs])
                assert torch.equal(k[b, h, i % bs], k0[a, h, j % bs])
                assert torch.equal(v[b, h, i % bs], v0[a, h, j % bs])
