"""GPU parity of pa_decode_tree against attention in 64 bits."""
import math

import pytest
import torch

from paged_kv_cache_251_gb300 import workloads as wl
from steplib import attention_bound, check_within, paged, random_parents, tree_oracle

pytestmark = pytest.mark.gpu


def run(q, k, v, tables, lens, mask, drafts, out_dtype, workspace=None, err=None, scale=None):
    from paged_kv_cache_251_gb300 import pa
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    pa.pa_decode_tree(out, q, k, v, tables, lens, tree_mask=mask, draft_lens=drafts, workspace=workspace,
                      err_word=err, scale=scale)
    return out


def check(q, k, v, tables, lens, drafts, mask, out_dtype, scale=None):
    T = q.shape[1]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(q, k, v, tables, lens, mask, drafts, out_dtype, err=err, scale=scale)
    d = drafts if drafts is not None else torch.full((q.shape[0],), T)
    ref, mag, dx = tree_oracle(q, k, v, tables, lens, d, mask, scale or 1 / math.sqrt(q.shape[-1]))
    torch.cuda.synchronize()
    assert err.item() == 0
    check_within(out, ref, attention_bound(ref, mag, dx, k.dtype, out_dtype, int(lens.max())))
    return out


CASES = [
    # H, H_kv, d, block, T, contexts (drafted tokens included), drafted
    (4, 4, 64, 16, 1, [1, 2, 17, 100], [1, 1, 1, 1]),
    (8, 2, 128, 16, 5, [5, 4, 0, 700], [5, 3, 0, 2]),                 # all drafted; an empty sequence
    (8, 1, 128, 8, 16, [16, 129, 1000], [16, 16, 9]),               # 128 rows a kv head
    (8, 2, 128, 16, 33, [33, 160, 515, 40], [33, 20, 33, 1]),        # 132 rows: two row tiles
    (16, 2, 64, 32, 40, [300, 41, 1025], [40, 40, 31]),
    (4, 4, 128, 32, 64, [64, 200], [64, 64]),
    (4, 2, 128, 16, 70, [500, 71], [70, 70]),                       # two mask words
    (2, 2, 64, 8, 130, [400, 131], [130, 100]),                       # three
    (8, 8, 128, 16, 8, [2048, 1111, 8, 9], [8, 8, 8, 8]),
    (8, 1, 128, 16, 64, [2000], [64]),                                # 512 rows
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("wide", [False, True])
def test_tree(case, dtype, wide):
    from paged_kv_cache_251_gb300 import pa
    h, hkv, d, bs, t, lens, drafted = case
    k, v, tables, lens_t = paged(17, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(9, 3, (len(lens), t, h, d), dtype=dtype).cuda()
    mask = pa.tree_mask_from_parents(random_parents(t, len(lens), t)).cuda()
    check(q, k, v, tables, lens_t, torch.tensor(drafted, dtype=torch.int32, device="cuda"), mask,
          torch.float32 if wide else dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_chain_is_causal_attention(dtype):
    """No mask and no drafted counts: a chain, every sequence with num_draft
    tokens; its last query equals pa_decode over the same context."""
    from paged_kv_cache_251_gb300 import pa
    lens, h, hkv, d, t = [40, 333, 6], 8, 2, 128, 6
    k, v, tables, lens_t = paged(3, lens, hkv, d, 16, dtype)
    q = wl.normal_tensor(8, 3, (3, t, h, d), dtype=dtype).cuda()
    out = check(q, k, v, tables, lens_t, None, None, torch.float32)
    one = torch.empty((3, h, d), device="cuda")
    pa.pa_decode(one, q[:, -1].contiguous(), k, v, tables, lens_t)
    torch.testing.assert_close(out[:, -1], one, rtol=2e-4, atol=2e-4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_masks_that_leave_a_row_empty(dtype, d):
    """No committed token and an empty mask row: zeros.  Full, empty and
    self-only rows side by side."""
    lens, t, h = [4, 70], 4, 8
    k, v, tables, lens_t = paged(5, lens, 2, d, 16, dtype)
    q = wl.normal_tensor(8, 3, (2, t, h, d), dtype=dtype).cuda()
    mask = torch.tensor([[[0], [15], [4], [-1]], [[0], [0], [8], [-1]]], dtype=torch.int64).cuda()
    out = check(q, k, v, tables, lens_t, None, mask, dtype)
    assert (out[0, 0] == 0).all()
    assert (out[1, 0] != 0).any()                # the committed tokens are still attended


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("h,t", [(8, 6), (8, 40)])
def test_non_finite_values_stay_in_their_place(dtype, bad, h, t):
    """K and V of a drafted token hold infinities or NaN: queries that do not
    attend it are untouched, those that do are not finite; the rows behind the
    context and the blocks of nobody hold NaN too."""
    from paged_kv_cache_251_gb300 import pa
    hkv, d, bs = 2, 128, 16
    lens = [t + 150, t + 3, 300]
    k, v, tables, lens_t = paged(6, lens, hkv, d, bs, dtype)
    used = torch.zeros(k.shape[0], bs, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        for tok in range(n):
            used[int(tables[s, tok // bs]), tok % bs] = True
    k.permute(0, 2, 1, 3)[~used] = float("nan")
    v.permute(0, 2, 1, 3)[~used] = float("nan")
    q = wl.normal_tensor(8, 3, (3, t, h, d), dtype=dtype).cuda()
    parents = random_parents(4, 3, t)
    mask = pa.tree_mask_from_parents(parents).cuda()
    clean = check(q, k, v, tables, lens_t, None, mask, dtype)
    j = 3
    hit = ((mask[:, :, 0] >> j) & 1).bool()
    for s, n in enumerate(lens):
        tok = n - t + j
        blk, row = int(tables[s, tok // bs]), tok % bs
        v[blk, :, row, 5] = bad
    out = run(q, k, v, tables, lens_t, mask, None, dtype)
    torch.cuda.synchronize()
    assert torch.equal(out[~hit], clean[~hit])
    same = [c for c in range(d) if c != 5]
    assert not torch.isfinite(out[hit][..., 5]).any()
    assert torch.isfinite(out[hit][..., same]).all()
    for s, n in enumerate(lens):
        tok = n - t + j
        k[int(tables[s, tok // bs]), :, tok % bs] = float("nan")
    out = run(q, k, v, tables, lens_t, mask, None, dtype)
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.isnan(out[hit]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_ramps_and_dominant_keys(dtype):
    """Scores that rise by 60 along the context (the running maximum moves in
    every tile), fall by 60, and one key far above the rest."""
    lens, t, h, hkv, d, bs = [900, 901, 650], 12, 8, 2, 128, 16
    k, v, tables, lens_t = paged(12, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(8, 3, (3, t, h, d), dtype=dtype).cuda()
    q[..., 0] = 8.0
    for s, n in enumerate(lens):
        tok = torch.arange(n, device="cuda")
        blk, row = tables[s, tok // bs].long(), tok % bs
        ramp = [60 * tok / n, 60 * (1 - tok / n), torch.where(tok == 77, 80.0, 0.0)][s]
        k[blk, :, row, 0] = (ramp * math.sqrt(d) / 8).to(dtype)[:, None]
    from paged_kv_cache_251_gb300 import pa
    mask = pa.tree_mask_from_parents(random_parents(2, 3, t)).cuda()
    for out_dtype in (torch.float32, dtype):
        check(q, k, v, tables, lens_t, None, mask, out_dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.3])
def test_scales(dtype, scale):
    """A negative scale, zero (the mean of V) and one larger than usual."""
    from paged_kv_cache_251_gb300 import pa
    lens, t, h, hkv, d = [300, 40], 20, 8, 2, 128
    k, v, tables, lens_t = paged(13, lens, hkv, d, 16, dtype)
    q = wl.normal_tensor(8, 3, (2, t, h, d), dtype=dtype).cuda()
    mask = pa.tree_mask_from_parents(random_parents(2, 2, t)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(q, k, v, tables, lens_t, mask, None, torch.float32, err=err, scale=scale)
    ref, mag, dx = tree_oracle(q, k, v, tables, lens_t, [t, t], mask, scale)
    assert err.item() == 0
    check_within(out, ref, attention_bound(ref, mag, dx, dtype, torch.float32, 300))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bad_tables_and_lengths(dtype):
    """Table entries outside the pool are left out and flagged; contexts beyond
    the table and drafted counts out of range are clamped and flagged."""
    from paged_kv_cache_251_gb300 import pa
    h, hkv, d, bs, t = 8, 2, 128, 16, 4
    lens = [400, 200, 64]
    k, v, tables, lens_t = paged(4, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(8, 3, (3, t, h, d), dtype=dtype).cuda()
    bad = tables.clone()
    bad[0, 3], bad[0, 4], bad[1, 0], bad[2, :] = -7, k.shape[0], 2 ** 31 - 1, -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(q, k, v, bad, lens_t, None, None, torch.float32, err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK
    assert (out[2] == 0).all()
    # the same with the tokens of those blocks never attended
    keep0 = [i for i in range(25) if i not in (3, 4)]
    t2 = torch.full_like(tables, -1)
    t2[0, :23] = tables[0, keep0]
    t2[1, :12] = tables[1, 1:13]
    l2 = torch.tensor([400 - 32, 200 - 16, 0], dtype=torch.int32, device="cuda")
    want = run(q, k, v, t2, l2, None, torch.tensor([4, 4, 0], dtype=torch.int32, device="cuda"), torch.float32)
    torch.testing.assert_close(out[:2], want[:2], rtol=1e-4, atol=1e-4)
    # lengths
    err.zero_()
    long = torch.tensor([400, 200, 10 ** 6], dtype=torch.int32, device="cuda")
    full = tables.clone()
    full[2] = tables[0]
    out = run(q, k, v, full, long, None, None, torch.float32, err=err)
    assert err.item() == pa.DEVERR_BAD_LEN
    long[2] = full.shape[1] * bs
    assert torch.equal(out, run(q, k, v, full, long, None, None, torch.float32))
    err.zero_()
    out = run(q, k, v, tables, lens_t, None, torch.tensor([9, -1, 4], dtype=torch.int32, device="cuda"),
              torch.float32, err=err)
    assert err.item() == pa.DEVERR_BAD_LEN
    assert (out[1] == 0).all()
    ok = run(q, k, v, tables, lens_t, None, torch.tensor([4, 0, 4], dtype=torch.int32, device="cuda"), torch.float32)
    assert torch.equal(out, ok)


def test_captured_replays_and_two_streams_match():
    """A captured call replayed on new inputs, and two calls at once on two
    streams with their own workspaces, give the bits of single calls."""
    from paged_kv_cache_251_gb300 import pa
    lens, h, hkv, d, t = [3000, 1700, 90, 2500], 8, 2, 128, 16
    k, v, tables, lens_t = paged(31, lens, hkv, d, 16, torch.bfloat16)
    mask = pa.tree_mask_from_parents(random_parents(4, 4, t)).cuda()
    qs = [wl.normal_tensor(40 + i, 3, (4, t, h, d), dtype=torch.bfloat16).cuda() for i in range(3)]
    want = [run(q, k, v, tables, lens_t, mask, None, torch.bfloat16) for q in qs]
    ws = [pa.tree_workspace_for(qs[0], k, tables.shape[1]) for _ in range(2)]
    q, out = qs[0].clone(), torch.empty_like(qs[0])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pa.pa_decode_tree(out, q, k, v, tables, lens_t, tree_mask=mask, workspace=ws[0])
    for i in (0, 1, 2, 1):
        q.copy_(qs[i])
        g.replay()
        assert torch.equal(out, want[i])
    outs = [torch.empty_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(2):
            pa.pa_decode_tree(outs[i], qs[i], k, v, tables, lens_t, tree_mask=mask, workspace=ws[i],
                              stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_same_bits_on_every_call():
    from paged_kv_cache_251_gb300 import pa
    lens, h, hkv, d, t = [5000, 100, 2047, 900], 16, 2, 128, 24
    k, v, tables, lens_t = paged(33, lens, hkv, d, 16, torch.float16)
    mask = pa.tree_mask_from_parents(random_parents(7, 4, t)).cuda()
    q = wl.normal_tensor(40, 3, (4, t, h, d), dtype=torch.float16).cuda()
    first = run(q, k, v, tables, lens_t, mask, None, torch.float32)
    for _ in range(10):
        assert torch.equal(run(q, k, v, tables, lens_t, mask, None, torch.float32), first)
