"""Serving-step operators at their edges: non-finite drafts across tiles, more
sequences than a grid dimension holds, repeated indices and slots, workspaces
with anything in them, a whole step captured and replayed."""
import math

import pytest
import torch

from paged_kv_cache_251_gb300 import workloads as wl
from steplib import attention_bound, check_within, paged, random_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,t", [(2, 1), (8, 24), (8, 60), (8, 140)])
@pytest.mark.parametrize("wide", [False, True])
def test_non_finite_drafts_across_tiles(dtype, d, h, t, wide):
    """Drafted tokens on both sides of a tile's end, several of them with an
    infinity, a negative one or a NaN in V: rows that attend none of them keep
    their bits on every call, the others get what they attend."""
    from paged_kv_cache_251_gb300 import pa
    hkv, bs = 2, 16
    lens = [256 + (t + 1) // 2, 128 + t - 1, 320 + t // 3, t]
    k, v, tables, lens_t = paged(t + d, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(8, 3, (4, t, h, d), dtype=dtype).cuda()
    mask = pa.tree_mask_from_parents(random_parents(t, 4, t)).cuda()
    out_dtype = torch.float32 if wide else dtype

    def run():
        out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
        return pa.pa_decode_tree(out, q, k, v, tables, lens_t, tree_mask=mask)

    clean = run()
    bad = {max(t // 2, 0): (float("inf"), 3), max(t - 2, 0): (float("-inf"), 7), t // 3: (float("nan"), 11)}
    hit = {c: torch.zeros((4, t), dtype=torch.bool, device="cuda") for c in (3, 7, 11)}
    for j, (x, c) in bad.items():
        for s, n in enumerate(lens):
            tok = n - t + j
            v[int(tables[s, tok // bs]), :, tok % bs, c] = x
        hit[c] |= ((mask[:, :, j // 64] >> (j % 64)) & 1).bool()
    want = clean.clone()
    for j, (x, c) in bad.items():
        want[hit[c]] = torch.where((torch.arange(d, device="cuda") == c), torch.tensor(x, dtype=out_dtype,
                                   device="cuda"), want[hit[c]])
    for _ in range(8):
        out = run()
        same = hit[3] | hit[7] | hit[11]
        assert torch.equal(out[~same], clean[~same])
        # (an attending row's finite columns may sum in another order: the poisoned tokens' terms come apart)
        assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
        assert torch.equal(out[torch.isinf(want)], want[torch.isinf(want)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_sequences_than_a_grid_dimension(dtype):
    """65600 short sequences over one small pool (blocks shared): decode of a
    drafted token, scored decode, selection and movement."""
    from paged_kv_cache_251_gb300 import pa
    N, d, bs, nb, scale = 65600, 64, 16, 50, 0.125
    k = wl.normal_tensor(1, 4, (nb, 1, bs, d), dtype=dtype).cuda()
    v = wl.normal_tensor(1, 5, (nb, 1, bs, d), dtype=dtype).cuda()
    tables = (wl.uniform01(2, 1, N) * nb).floor().to(torch.int32).view(N, 1).cuda()
    lens = (wl.uniform01(3, 1, N) * (bs + 1)).floor().to(torch.int32).cuda()
    q = wl.normal_tensor(4, 3, (N, 1, d), dtype=dtype).cuda()
    kr, vr = k[tables[:, 0].long(), 0].double(), v[tables[:, 0].long(), 0].double()
    live = torch.arange(bs, device="cuda") < lens[:, None]
    x = (kr @ q[:, 0, :, None].double())[..., 0] * scale
    w = torch.softmax(x.masked_fill(~live, float("-inf")), -1).nan_to_num(0.0)
    ref, mag = (w[:, None] @ vr), (w[:, None] @ vr.abs())
    dx = ((kr.abs() @ q[:, 0, :, None].double().abs())[..., 0] * live * scale).amax(-1, True) * (d + 2) * 2.0 ** -24
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bound = attention_bound(ref, mag, dx, dtype, torch.float32, bs)
    out = torch.full((N, 1, 1, d), float("nan"), device="cuda")
    pa.pa_decode_tree(out, q.view(N, 1, 1, d), k, v, tables, lens, draft_lens=lens.clamp_max(1), err_word=err,
                      scale=scale)
    check_within(out.view(N, 1, d), ref, bound, "tree")
    out = torch.full((N, 1, d), float("nan"), device="cuda")
    sc = torch.full((N, 1, bs), -1.0, device="cuda")
    pa.pa_decode_scored(out, sc, q, k, v, tables, lens, scale=scale, err_word=err)
    # a weight: exp of a score off by dx twice over (numerator and denominator), the
    # exponentials' and the sums' roundings
    check_within(torch.where(live, sc[:, 0], 0.0), w,
                 w * (2 * dx + 2 * (2.0 ** -21 + 2.0 ** -17) + (bs + 4) * 2.0 ** -24) + 2.0 ** -126, "scores")
    assert (sc[:, 0][~live] == -1).all()
    keep = torch.empty((N, 1, 6), dtype=torch.int32, device="cuda")
    new = torch.empty(N, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new, None, sc, lens, 6, 2, err_word=err)
    assert torch.equal(new, lens.clamp_max(6))
    last = torch.arange(bs, device="cuda") >= (lens - 2)[:, None]
    rank = torch.where(live, torch.where(last, 9.0, sc[:, 0]), -1.0)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :6].sort(-1).values.to(torch.int32)
    longer = lens > 6
    assert torch.equal(keep[longer, 0], order[longer])
    short = torch.arange(6, device="cuda", dtype=torch.int32)
    assert torch.equal(keep[~longer, 0], torch.where(short < lens[~longer, None], short, -1))
    # into one block a sequence
    k2 = torch.cat([k, torch.zeros((N, 1, bs, d), dtype=dtype, device="cuda")])
    v2 = torch.cat([v, torch.zeros((N, 1, bs, d), dtype=dtype, device="cuda")])
    dst = torch.arange(nb, nb + N, dtype=torch.int32, device="cuda").view(N, 1)
    pa.pa_compact_kv(k2, v2, keep, new, tables, dst_block_tables=dst, err_word=err)
    assert err.item() == 0 and torch.equal(k2[:nb], k) and torch.equal(v2[:nb], v)
    at = keep[:, 0].clamp_min(0).long()
    on = (short < new[:, None])[..., None]
    for got, rows in ((k2, kr), (v2, vr)):
        want = torch.where(on, rows.gather(1, at[..., None].expand(-1, -1, d)), 0.0).to(dtype)
        assert torch.equal(got[nb:, 0, :6], want) and (got[nb:, 0, 6:] == 0).all()


def test_repeated_indices_and_slots():
    """In place, kept indices at or above their places in any order and more than
    once; a slot named by many tokens (not allowed) holds elements of theirs, and
    nothing else is touched."""
    from paged_kv_cache_251_gb300 import pa
    d, bs, n = 128, 16, 700
    k, v, tables, _ = paged(7, [n], 2, d, bs, torch.float16)
    i = torch.arange(600)
    keep = torch.minimum(i + (wl.uniform01(5, 1, 600) * 100).floor().long(), torch.tensor(n - 1)).to(torch.int32)
    rows = lambda c: c[tables[0].long()].transpose(1, 2).reshape(-1, 2, d)[:n].clone()  # noqa: E731
    k0, v0 = rows(k), rows(v)
    pa.pa_compact_kv(k, v, keep.view(1, 1, -1).cuda(), torch.tensor([600], dtype=torch.int32, device="cuda"), tables)
    for c, c0 in ((k, k0), (v, v0)):
        assert torch.equal(rows(c)[:600], c0[keep.long().cuda()]) and torch.equal(rows(c)[600:], c0[600:])
    x = wl.normal_tensor(3, 3, (40, 2, d), dtype=torch.float16).cuda()
    kc, vc = torch.zeros((4, 2, bs, d), dtype=torch.float16, device="cuda"), torch.zeros((4, 2, bs, d),
                                                                                     dtype=torch.float16, device="cuda")
    pa.pa_rope_append_kv(torch.empty_like(x), x, x, x, torch.zeros(40, dtype=torch.int32, device="cuda"),
                         torch.full((40,), 21, dtype=torch.int64, device="cuda"), pa.pa_rope_frequencies(d).cuda(), kc,
                         vc)
    for c in (kc, vc):
        for head in range(2):
            assert (x[:, head] == c[1, head, 5]).any(0).all()
        c[1, :, 5] = 0
        assert (c == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_captured_step_replays_on_new_inputs(dtype):
    """Rotate and append drafts, check the tree, commit, decode with scores,
    select and move, all in one graph on a side stream; workspaces full of NaN.
    Replays on other inputs give the bits of the same calls made one by one."""
    from paged_kv_cache_251_gb300 import pa
    N, T, h, hkv, d, bs = 3, 6, 8, 2, 128, 16
    lens = [400, 33, 1300]
    k0, v0, tables, _ = paged(51, [n + T for n in lens], hkv, d, bs, dtype, extra_blocks=30)
    used = set(tables[tables >= 0].tolist())
    free = [b for b in range(k0.shape[0]) if b not in used]
    budget = 128
    dst = torch.tensor(free[:N * 8], dtype=torch.int32, device="cuda").view(N, 8)
    base = torch.tensor(lens, dtype=torch.int32, device="cuda")
    full = base + T
    slots = torch.tensor([int(tables[s, (n + j) // bs]) * bs + (n + j) % bs for s, n in enumerate(lens)
                          for j in range(T)], dtype=torch.int64, device="cuda")
    pos = torch.tensor([n + j for n in lens for j in range(T)], dtype=torch.int32, device="cuda")
    f = pa.pa_rope_frequencies(d).cuda()
    mask = pa.tree_mask_from_parents(random_parents(4, N, T)).cuda()
    took = torch.tensor([[[0, 2, 5]], [[1, 1, 1]], [[0, 1, 4]]], dtype=torch.int32, device="cuda")
    ntook = torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda")
    inputs = [wl.normal_tensor(60 + i, 3, (N * T, (h + 2 * hkv) * d), dtype=dtype).cuda() for i in range(3)]
    qkv, kc, vc = inputs[0].clone(), k0.clone(), v0.clone()
    width = tables.shape[1] * bs
    new_len = base + ntook
    bufs = dict(q=torch.empty((N, T, h, d), dtype=dtype, device="cuda"),
                out=torch.empty((N, T, h, d), dtype=dtype, device="cuda"),
                last=torch.empty((N, h, d), dtype=dtype, device="cuda"),
                sc=torch.empty((N, hkv, width), device="cuda"),
                keep=torch.empty((N, hkv, budget), dtype=torch.int32, device="cuda"),
                n=torch.empty(N, dtype=torch.int32, device="cuda"),
                err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    tree_ws = pa.tree_workspace_for(bufs["q"], kc, tables.shape[1])
    scored_ws = pa.scored_workspace_for(bufs["last"], kc, tables.shape[1])
    first = torch.zeros((N, hkv, width), device="cuda")

    def step(stream=None):
        q = qkv[:, :h * d].view(N * T, h, d)
        k = qkv[:, h * d:(h + hkv) * d].view(N * T, hkv, d)
        v = qkv[:, (h + hkv) * d:].view(N * T, hkv, d)
        e = bufs["err"]
        pa.pa_rope_append_kv(bufs["q"].view(N * T, h, d), q, k, v, pos, slots, f, kc, vc, err_word=e, stream=stream)
        pa.pa_decode_tree(bufs["out"], bufs["q"], kc, vc, tables, full, tree_mask=mask, workspace=tree_ws, err_word=e,
                          stream=stream)
        pa.pa_compact_kv(kc, vc, took, ntook, tables, base_lens=base, err_word=e, stream=stream)
        pa.pa_decode_scored(bufs["last"], bufs["sc"], bufs["q"].view(N * T, h, d)[:N], kc, vc, tables, new_len,
                            scores_in=first, workspace=scored_ws, err_word=e, stream=stream)
        pa.pa_evict_select(bufs["keep"], bufs["n"], bufs["sc"], bufs["sc"], new_len, budget, 16, err_word=e,
                           stream=stream)
        pa.pa_compact_kv(kc, vc, bufs["keep"], bufs["n"], tables, dst_block_tables=dst, err_word=e, stream=stream)

    def reset(i):
        qkv.copy_(inputs[i])
        kc.copy_(k0)
        vc.copy_(v0)
        bufs["sc"].zero_()
        for ws in (tree_ws, scored_ws):
            if ws is not None:
                ws.fill_(float("nan"))

    def results():
        torch.cuda.synchronize()
        return {**{n: t.clone() for n, t in bufs.items()}, "k": kc.clone(), "v": vc.clone()}

    want = []
    for i in range(3):
        reset(i)
        step()
        want.append(results())
        assert want[i]["err"].item() == 0 and want[i]["n"].tolist() == [128, 34, 128]
        assert torch.isfinite(want[i]["out"]).all() and torch.isfinite(want[i]["sc"]).all()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in (0, 2, 1, 2):
        reset(i)
        torch.cuda.synchronize()
        g.replay()
        got = results()
        for name, t in got.items():
            assert torch.equal(t, want[i][name]), (i, name)
    reset(1)
    torch.cuda.synchronize()
    step(stream=side)
    got = results()
    for name, t in got.items():
        assert torch.equal(t, want[1][name]), name


def test_empty_batches():
    """No sequence or no token: nothing is launched, nothing refused."""
    from paged_kv_cache_251_gb300 import pa
    i32 = dict(dtype=torch.int32, device="cuda")
    kc = torch.zeros((2, 2, 16, 64), device="cuda")
    none = torch.empty((0, 2, 64), device="cuda")
    f = pa.pa_rope_frequencies(64).cuda()
    pos, lens, tables = torch.empty(0, **i32), torch.empty(0, **i32), torch.empty((0, 4), **i32)
    pa.pa_rope(none, none, pos, f)
    pa.pa_rope_append_kv(none, none, none, none, pos, torch.empty(0, dtype=torch.int64, device="cuda"), f, kc, kc)
    pa.pa_decode_tree(torch.empty((0, 3, 2, 64), device="cuda"), torch.empty((0, 3, 2, 64), device="cuda"), kc, kc,
                      tables, lens)
    pa.pa_decode_scored(none, torch.empty((0, 2, 64), device="cuda"), none, kc, kc, tables, lens)
    pa.pa_evict_select(torch.empty((0, 2, 5), **i32), lens, None, torch.empty((0, 2, 64), device="cuda"), lens, 5, 1)
    pa.pa_compact_kv(kc, kc.clone(), torch.empty((0, 1, 5), **i32), lens, tables)
    pa.pa_compact_kv(kc, kc.clone(), torch.empty((1, 1, 0), **i32), torch.zeros(1, **i32), torch.zeros((1, 4), **i32))
    torch.cuda.synchronize()
    assert (kc == 0).all() and math.isfinite(float(kc.sum()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("h,hkv,d,rot,inter", [(1, 1, 64, 64, True), (2, 1, 128, 2, False), (3, 1, 64, 48, False),
                                               (70, 35, 64, 64, False)])
def test_many_tokens_a_block_of_threads(dtype, h, hkv, d, rot, inter):
    """Few heads: up to eight tokens a CTA, the last one ragged; a row that needs
    nearly all threads of a CTA; more rows a token than a CTA holds at once."""
    from paged_kv_cache_251_gb300 import pa
    from test_gpu_rope import check, rotate64
    n, bs = 12003 if h < 10 else 1500, 16
    q = wl.normal_tensor(1, 3, (n, h, d), dtype=dtype).cuda()
    k = wl.normal_tensor(2, 3, (n, hkv, d), dtype=dtype).cuda()
    v = wl.normal_tensor(3, 3, (n, hkv, d), dtype=dtype).cuda()
    freqs = pa.pa_rope_frequencies(rot)
    pos = wl.randint(7, 1, n, 0, 100000).to(torch.int32).cuda()
    nb = (n + bs - 1) // bs
    slots = wl.permutation(5, 2, nb * bs)[:n].cuda()
    kc = torch.zeros((nb, hkv, bs, d), dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    out = torch.full_like(q, float("nan"))
    pa.pa_rope_append_kv(out, q, k, v, pos, slots, freqs.cuda(), kc, vc, interleaved=inter)
    ref, mag = rotate64(q, pos, freqs, rot, inter, 1.0)
    check(out, ref, mag, 1.0, 1e5)
    ref, mag = rotate64(k, pos, freqs, rot, inter, 1.0)
    check(kc.transpose(1, 2).reshape(nb * bs, hkv, d)[slots], ref, mag, 1.0, 1e5)
    assert torch.equal(vc.transpose(1, 2).reshape(nb * bs, hkv, d)[slots], v)


@pytest.mark.parametrize("L,budget,recent", [(5000, 4999, 0), (33333, 1, 0), (33333, 700, 700), (60001, 20000, 1),
                                             (20000, 20000, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_select_of_special_values_over_slices(L, budget, recent, in_place):
    """Infinities, NaN, zeros of both signs and subnormals in rows shared by several
    CTAs, off the 16-byte boundary; budgets of one, of nearly all, of only recent
    tokens."""
    from paged_kv_cache_251_gb300 import pa
    from test_gpu_evict import select_oracle
    values = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-42, -1e-42, 1.0, 3.5, -2.0, 0.7,
                           0.71])
    sc = values[(wl.uniform01(L + budget, 1, 2 * (L + 1)) * 12).floor().long()].view(1, 2, L + 1).contiguous()
    dev = sc.cuda()
    out = dev if in_place else torch.full_like(dev, 9.0)
    keep = torch.empty((1, 2, budget), dtype=torch.int32, device="cuda")
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new, out, dev, torch.tensor([L], dtype=torch.int32, device="cuda"), budget, recent)
    want, n, scores = select_oracle(sc, [L], budget, recent)
    assert new.tolist() == [min(L, budget)] and torch.equal(keep.cpu(), want)
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=1.5), torch.nan_to_num(scores, nan=1.5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv,t", [(1, 1, 1), (2, 1, 3), (4, 1, 9), (4, 1, 64), (8, 1, 100)])
@pytest.mark.parametrize("wide", [False, True])
def test_one_long_context_in_many_parts(dtype, d, h, hkv, t, wide):
    """A context cut into about 150 parts, from one row to 800: the merge shares a
    pair's columns among all CTAs, or its parts among warps; and a second sequence
    of one tile beside it."""
    from paged_kv_cache_251_gb300 import pa
    from steplib import tree_oracle
    lens = [30011, t]
    k, v, tables, lens_t = paged(t + h, lens, hkv, d, 32, dtype)
    q = wl.normal_tensor(8, 3, (2, t, h, d), dtype=dtype).cuda()
    mask = pa.tree_mask_from_parents(random_parents(t, 2, t)).cuda()
    drafts = torch.tensor([max(t - 1, 1), t], dtype=torch.int32, device="cuda")
    out_dtype = torch.float32 if wide else dtype
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_decode_tree(out, q, k, v, tables, lens_t, tree_mask=mask, draft_lens=drafts, err_word=err)
    ref, mag, dx = tree_oracle(q, k, v, tables, lens_t, drafts, mask, 1 / math.sqrt(d))
    assert err.item() == 0
    check_within(out, ref, attention_bound(ref, mag, dx, dtype, out_dtype, max(lens)))
    # rows that are padding are zero
    assert t == 1 or (out[0, t - 1] == 0).all()
