"""Tree attention where a CTA has many items: drafted tokens with non-finite V
rows in some sequences, whose neighbours keep their bits."""
import pytest
import torch

from paged_kv_cache_251_gb300 import workloads as wl
from steplib import paged, random_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,h", [(3, 4), (16, 16), (24, 16)])     # 6 and 128 rows a kv head, and 192
@pytest.mark.parametrize("every", [2, 3])
def test_neighbours_of_non_finite_drafts_keep_their_bits(dtype, t, h, every):
    """600 sequences of one or two tiles, two kv heads: eight items a CTA.  Every
    second or third has a drafted token with an infinity in V, in the first tile
    or the second; the others give the bits of the call without them, and those
    queries that attend it are not finite, on repeated calls."""
    from paged_kv_cache_251_gb300 import pa
    hkv, d, bs, n_seqs = 2, 128, 16, 600
    lens = [t + (7 * s) % (250 - t) for s in range(n_seqs)]
    k, v, tables, lens_t = paged(41, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(42, 3, (n_seqs, t, h, d), dtype=dtype).cuda()
    mask = pa.tree_mask_from_parents(random_parents(43, n_seqs, t)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pa.tree_workspace_for(q, k, tables.shape[1])

    def run():
        out = torch.empty_like(q)
        return pa.pa_decode_tree(out, q, k, v, tables, lens_t, tree_mask=mask, workspace=ws, err_word=err)

    clean = run()
    bad = torch.arange(n_seqs, device="cuda") % every == 1
    tok = lens_t.long() - t + 1
    at = bad.nonzero()[:, 0]
    v[tables[at, tok[at] // bs].long(), :, tok[at] % bs, 9] = float("inf")
    hit = ((mask[:, :, 0] >> 1) & 1).bool() & bad[:, None]
    for _ in range(20):
        out = run()
        assert torch.equal(out[~hit], clean[~hit])
        assert not torch.isfinite(out[hit][..., 9]).any()
        assert torch.isfinite(out[hit][..., :9]).all() and torch.isfinite(out[hit][..., 10:]).all()
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("drafted", [1, 8, 16, 20])
def test_rows_behind_the_context_where_warps_have_no_row(dtype, drafted):
    """Two row tiles (24 tokens x 8 heads) with few drafted: warps without a live row
    still zero the V rows behind the context, which hold NaN here."""
    from paged_kv_cache_251_gb300 import pa
    t, h, hkv, d, bs, n_seqs = 24, 16, 2, 128, 32, 60
    lens = [drafted + (5 * s) % 200 for s in range(n_seqs)]
    k, v, tables, lens_t = paged(44, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(45, 3, (n_seqs, t, h, d), dtype=dtype).cuda()
    drafts = torch.full((n_seqs,), drafted, dtype=torch.int32, device="cuda")
    ws = pa.tree_workspace_for(q, k, tables.shape[1])

    def run():
        out = torch.full_like(q, float("nan"))
        return pa.pa_decode_tree(out, q, k, v, tables, lens_t, draft_lens=drafts, workspace=ws)

    last = tables.gather(1, ((lens_t.long() - 1) // bs)[:, None])[:, 0].long()
    behind = torch.arange(bs, device="cuda") > ((lens_t - 1) % bs)[:, None]
    rows = v.permute(0, 2, 1, 3)
    held = rows[last]
    rows[last] = torch.where(behind[:, :, None, None], torch.zeros_like(held), held)
    clean = run()
    assert torch.isfinite(clean).all()
    rows[last] = torch.where(behind[:, :, None, None], torch.full_like(held, float("nan")), held)
    for _ in range(20):
        assert torch.equal(run(), clean)
