"""GPU parity of pa_decode_scored, pa_evict_select and pa_compact_kv."""
import math

import pytest
import torch

from paged_kv_cache_251_gb300 import workloads as wl
from steplib import U32, attend, attention_bound, check_within, paged, rows_of

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# scored decode

SCORED = [
    # H, H_kv, d, block, contexts, partition
    (4, 4, 64, 16, [1, 2, 17, 100], 0),
    (5, 5, 128, 8, [0, 700, 33], 0),
    (8, 8, 128, 32, [3000, 1], 256),
    (8, 2, 128, 16, [1500, 16, 0, 129], 128),
    (8, 4, 128, 8, [64, 1025], 0),
    (16, 2, 128, 32, [2500, 31], 512),
    (8, 2, 64, 16, [900, 5], 128),
    (8, 1, 64, 8, [77], 0),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", SCORED)
@pytest.mark.parametrize("inputs", ["in", "none", "same"])
def test_scored_decode(case, dtype, inputs):
    from paged_kv_cache_251_gb300 import pa
    h, hkv, d, bs, lens, part = case
    N, G = len(lens), h // hkv
    k, v, tables, lens_t = paged(21, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(9, 3, (N, h, d), dtype=dtype).cuda()
    width = tables.shape[1] * bs + 5                     # a stride of its own
    given = torch.rand((N, hkv, width), device="cuda") * 3
    out = torch.full((N, h, d), float("nan"), device="cuda")
    dst = given.clone() if inputs == "same" else torch.full_like(given, -7.0)
    before = dst.clone()
    src = {"in": given, "none": None, "same": dst}[inputs]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_decode_scored(out, dst, q, k, v, tables, lens_t, scores_in=src, partition_size=part, err_word=err)
    plain = torch.empty_like(out)
    pa.pa_decode(plain, q, k, v, tables, lens_t, partition_size=part)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert torch.equal(out, plain)                       # pa_decode's own result
    base = torch.zeros_like(given) if inputs == "none" else given
    for s, n in enumerate(lens):
        kk, vv = rows_of(k, tables[s], n), rows_of(v, tables[s], n)
        ref, mag, dx, w = attend(q[s].double().view(1, hkv, G, d), kk, vv,
                                 torch.ones((1, n), dtype=torch.bool, device="cuda"), 1 / math.sqrt(d))
        want = base[s, :, :n].double() + w[0].sum(1)
        # a weight moves by 2 dx relative with its row's scores, plus the exponentials (argument below 2^7 in
        # base-2 units) and the denominators' sums; then the fp32 additions
        slack = (w[0] * (2 * dx[0][..., None] + 2 ** -20 + 2 ** 8 * U32 + math.sqrt(max(n, 1)) * 2 * U32)).sum(1)
        bound = slack + (want.abs() + w[0].sum(1)) * (G + 1) * U32 + 1e-12
        assert ((dst[s, :, :n].double() - want).abs() <= bound).all()
        assert torch.equal(dst[s, :, n:], before[s, :, n:])   # behind the context: left as it was
        if n:
            # each row's weights sum to one
            total = dst[s, :, :n].double().sum(-1) - base[s, :, :n].double().sum(-1)
            assert ((total - G).abs() <= float(bound.sum(-1).max())).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("h,hkv,d", [(4, 4, 128), (8, 2, 128), (8, 2, 64)])
def test_scored_decode_with_bad_blocks(dtype, h, hkv, d):
    """Tokens behind a bad table entry get no weight; the error word tells."""
    from paged_kv_cache_251_gb300 import pa
    lens, bs = [300, 100], 16
    k, v, tables, lens_t = paged(22, lens, hkv, d, bs, dtype)
    q = wl.normal_tensor(9, 3, (2, h, d), dtype=dtype).cuda()
    tables[0, 2], tables[1, :] = -1, k.shape[0]
    out, sc = torch.empty((2, h, d), device="cuda"), torch.full((2, hkv, tables.shape[1] * bs), 5.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_decode_scored(out, sc, q, k, v, tables, lens_t, partition_size=128, err_word=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK
    assert (sc[0, :, 32:48] == 0).all() and (sc[1, :, :100] == 0).all() and (out[1] == 0).all()
    assert (sc[0, :, :32] > 0).all() and (sc[0, :, 48:300] > 0).all()
    assert ((sc[0, :, :300].sum(-1) - h // hkv).abs() < 1e-4).all()
    assert (sc[:, :, 304:] == 5.0).all()


def test_scored_decode_twice_gives_the_same_bits_and_replays():
    from paged_kv_cache_251_gb300 import pa
    lens, h, hkv, d, bs = [3000, 1200, 40, 2047], 8, 2, 128, 16
    k, v, tables, lens_t = paged(23, lens, hkv, d, bs, torch.bfloat16)
    q = wl.normal_tensor(9, 3, (4, h, d), dtype=torch.bfloat16).cuda()
    sc = torch.zeros((4, hkv, tables.shape[1] * bs), device="cuda")
    out, ws = torch.empty_like(q), pa.scored_workspace_for(q, k, tables.shape[1])
    first = sc.clone()
    pa.pa_decode_scored(out, first, q, k, v, tables, lens_t, workspace=ws)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pa.pa_decode_scored(out, sc, q, k, v, tables, lens_t, scores_in=sc, workspace=ws)
    for _ in range(3):
        g.replay()
    assert torch.equal(out, want)
    assert torch.equal(sc, first + first + first)


# ---------------------------------------------------------------------------
# selection


def select_oracle(scores, lens, budget, recent):
    """(keep, new_lens, scores_out) by sorting each row in Python."""
    N, K, W = scores.shape
    keep = torch.full((N, K, budget), -1, dtype=torch.int32)
    out = torch.zeros((N, K, W))
    new = []
    sc = scores.cpu()
    for s, n in enumerate(lens):
        new.append(min(n, budget))
        for h in range(K):
            row = sc[s, h].tolist()
            if n <= budget:
                chosen = list(range(n))
            else:
                rank = sorted(range(n - recent), key=lambda t: (not math.isnan(row[t]), -row[t] if row[t] == row[t]
                                                                else 0.0, t))
                chosen = sorted(rank[:budget - recent]) + list(range(n - recent, n))
            keep[s, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            out[s, h, :len(chosen)] = sc[s, h, chosen]
    return keep, torch.tensor(new, dtype=torch.int32), out


SELECT = [
    # kv heads, contexts, budget, recent
    (1, [1], 1, 0),
    (1, [2, 1, 0], 1, 1),
    (4, [100, 31, 32, 33, 0], 32, 8),
    (2, [513, 512, 511, 1025], 512, 0),
    (2, [700, 699], 64, 64),                 # recent only
    (3, [5000, 2049], 2048, 100),
    (1, [40000], 33, 7),
]


@pytest.mark.parametrize("case", SELECT)
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special"])
@pytest.mark.parametrize("in_place", [False, True])
def test_select(case, kind, in_place):
    from paged_kv_cache_251_gb300 import pa
    K, lens, budget, recent = case
    N, W = len(lens), max(max(lens), 1) + 3
    sc = wl.normal_tensor(sum(lens), 3, (N, K, W)).abs()
    if kind == "ties":
        sc = (sc * 4).round() / 4
    elif kind == "equal":
        sc = torch.full_like(sc, 0.5)
    elif kind == "special":
        u = wl.uniform01(3, 1, sc.numel()).view(sc.shape)
        sc[u < 0.1] = 0.0
        sc[(u > 0.1) & (u < 0.2)] = -0.0
        sc[(u > 0.2) & (u < 0.22)] = float("inf")
        sc[(u > 0.3) & (u < 0.32)] = float("nan")
        sc[(u > 0.4) & (u < 0.5)] *= -1
        sc[(u > 0.5) & (u < 0.52)] = float("-inf")
        sc[(u > 0.6) & (u < 0.7)] *= 1e-40
    dev = sc.cuda()
    out = dev if in_place else torch.full_like(dev, 9.0)
    keep = torch.full((N, K, budget), 77, dtype=torch.int32, device="cuda")
    new = torch.full((N,), 77, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new, out, dev, lens_t, budget, recent, err_word=err)
    k_ref, n_ref, s_ref = select_oracle(sc, lens, budget, recent)
    assert err.item() == 0
    assert torch.equal(new.cpu(), n_ref)
    assert torch.equal(keep.cpu(), k_ref)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(s_ref))
    assert torch.equal(torch.nan_to_num(got, nan=1.5), torch.nan_to_num(s_ref, nan=1.5))


@pytest.mark.parametrize("L", [3000, 70001, 400003])
@pytest.mark.parametrize("in_place", [False, True])
def test_select_over_slices(L, in_place):
    """Rows shared by several CTAs, and one beyond what they hold: many ties around
    the cut, against a stable sort."""
    from paged_kv_cache_251_gb300 import pa
    K, budget, recent = 2, L // 3, 17
    sc = (wl.normal_tensor(L, 3, (1, K, L)).abs() * 8).round() / 8
    dev = sc.cuda()
    out = dev if in_place else torch.full_like(dev, 9.0)
    keep = torch.empty((1, K, budget), dtype=torch.int32, device="cuda")
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new, out, dev, torch.tensor([L], dtype=torch.int32, device="cuda"), budget, recent)
    for h in range(K):
        order = torch.sort(sc[0, h, :L - recent], descending=True, stable=True).indices[:budget - recent]
        want = torch.cat([order.sort().values, torch.arange(L - recent, L)])
        assert torch.equal(keep[0, h].cpu().long(), want)
        assert torch.equal(out[0, h, :budget].cpu(), sc[0, h, want]) and (out[0, h, budget:] == 0).all()


def test_select_clamps_long_contexts_and_writes_no_scores_when_asked():
    from paged_kv_cache_251_gb300 import pa
    sc = torch.rand((2, 2, 50), device="cuda")
    keep = torch.empty((2, 2, 10), dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new, None, sc, torch.tensor([51, -3], dtype=torch.int32, device="cuda"), 10, 2,
                       err_word=err)
    assert err.item() == pa.DEVERR_BAD_LEN
    want, _, _ = select_oracle(sc, [50, 0], 10, 2)
    assert torch.equal(keep.cpu(), want) and new.tolist() == [10, 0]


# ---------------------------------------------------------------------------
# movement


def compact_oracle(k, tables, dst_tables, keep, keep_lens, base):
    """Row by row on a copy; the source rows are those before the call."""
    out, bs = k.clone(), k.shape[2]
    for s in range(keep.shape[0]):
        for h in range(k.shape[1]):
            for i in range(int(keep_lens[s])):
                j = int(keep[s, h if keep.shape[1] > 1 else 0, i])
                a, b = int(base[s]) + j, int(base[s]) + i
                out[int(dst_tables[s, b // bs]), h, b % bs] = k[int(tables[s, a // bs]), h, a % bs]
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("where", ["in place", "other blocks", "other table width"])
@pytest.mark.parametrize("heads", [1, 3])
def test_compact(dtype, d, bs, where, heads):
    from paged_kv_cache_251_gb300 import pa
    lens, base, K = [700, 1, 40, 0, 257], [0, 0, 30, 0, 100], 3
    extra = 200 // bs * 8
    k, v, tables, _ = paged(41, lens, K, d, bs, dtype, extra_blocks=extra, device="cpu")
    used = set(tables[tables >= 0].tolist())
    free = [b for b in range(k.shape[0]) if b not in used]
    counts = [300, 1, 7, 0, 157]
    keep = torch.full((5, heads, 300), -1, dtype=torch.int32)
    for s, c in enumerate(counts):
        for h in range(heads):
            keep[s, h, :c] = wl.permutation(s * 7 + h, 2, lens[s] - base[s])[:c].sort().values.to(torch.int32)
    dst = None
    if where != "in place":
        width = tables.shape[1] if where == "other blocks" else (300 + bs - 1) // bs
        dst = torch.full((5, width), -1, dtype=torch.int32)
        for s, c in enumerate(counts):
            for b in range(base[s] // bs, (base[s] + c + bs - 1) // bs):
                dst[s, b] = free.pop()
    base_t = torch.tensor(base, dtype=torch.int32)
    counts_t = torch.tensor(counts, dtype=torch.int32)
    kd, vd = k.cuda(), v.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_compact_kv(kd, vd, keep.cuda(), counts_t.cuda(), tables.cuda(),
                     dst_block_tables=None if dst is None else dst.cuda(), base_lens=base_t.cuda(), err_word=err)
    assert err.item() == 0
    to = tables if dst is None else dst
    assert torch.equal(kd.cpu(), compact_oracle(k, tables, to, keep, counts, base))
    assert torch.equal(vd.cpu(), compact_oracle(v, tables, to, keep, counts, base))


def test_compact_bad_indices_and_tables():
    """Indices below their place (in place), beyond the table or negative, bad
    table entries and places past the destination move nothing and are flagged;
    counts are clamped to the list."""
    from paged_kv_cache_251_gb300 import pa
    d, bs, K = 64, 8, 2
    k, v, tables, _ = paged(42, [40, 40, 40], K, d, bs, torch.float32, extra_blocks=12, device="cpu")
    keep = torch.tensor([[[2, 0, 5, 40]], [[-1, 3, 9, 39]], [[0, 2, 17, 25]]], dtype=torch.int32)
    bad = tables.clone()
    bad[2, 2] = k.shape[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kd, vd = k.cuda(), v.cuda()
    n = torch.tensor([4, 99, 4], dtype=torch.int32)
    pa.pa_compact_kv(kd, vd, keep.cuda(), n.cuda(), bad.cuda(), err_word=err)
    assert err.item() == pa.DEVERR_BAD_INDEX | pa.DEVERR_BAD_BLOCK
    fine = [(0, 0, 2), (0, 2, 5), (1, 1, 3), (1, 2, 9), (1, 3, 39), (2, 1, 2), (2, 3, 25)]
    want = k.clone()
    for s, i, j in fine:
        want[int(tables[s, i // bs]), :, i % bs] = k[int(tables[s, j // bs]), :, j % bs]
    assert torch.equal(kd.cpu(), want)
    # other blocks, a destination table of one block: places from 8 on have none
    err.zero_()
    dst = torch.tensor([[k.shape[0] - 1], [-1], [0]], dtype=torch.int32)
    used = set(tables[tables >= 0].tolist())
    free = [b for b in range(k.shape[0]) if b not in used]
    dst[0, 0], dst[2, 0] = free[0], free[1]
    keep = torch.arange(12, dtype=torch.int32).flip(0).view(1, 1, 12).repeat(3, 1, 1).contiguous()
    kd, vd = k.cuda(), v.cuda()
    pa.pa_compact_kv(kd, vd, keep.cuda(), torch.full((3,), 12, dtype=torch.int32).cuda(), tables.cuda(),
                     dst_block_tables=dst.cuda(), err_word=err)
    assert err.item() == pa.DEVERR_BAD_INDEX | pa.DEVERR_BAD_BLOCK
    want = k.clone()
    for s in (0, 2):
        for i in range(8):
            want[int(dst[s, 0]), :, i] = k[int(tables[s, (11 - i) // bs]), :, (11 - i) % bs]
    assert torch.equal(kd.cpu(), want)


# ---------------------------------------------------------------------------
# together


def test_serving_steps_with_drafts_and_eviction():
    """Steps of a small serving loop on two sequences: rotate and append the
    prompt, draft a tree (rotate + append), check it, commit the accepted path
    (in place), decode with scores, evict into renewed blocks, decode again;
    each result against a model that keeps every head's rows in plain lists."""
    from paged_kv_cache_251_gb300 import pa
    from paged_kv_cache_251_gb300.blocks import BlockManager
    N, h, hkv, d, bs, dtype = 2, 8, 2, 128, 16, torch.bfloat16
    nb, M = 64, 24
    bm = BlockManager(nb, bs, N, M, free_order=wl.permutation(3, 2, nb))
    kc = torch.zeros((nb, hkv, bs, d), dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    f = pa.pa_rope_frequencies(d).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = [[[] for _ in range(hkv)] for _ in range(N)]     # (k, v) rows per sequence and kv head
    seed = [100]

    def tokens(counts, positions):
        """Append counts[s] new tokens with these positions; returns their rotated queries."""
        seqs = [s for s in range(N) for _ in range(counts[s])]
        slots, pairs = bm.append(seqs)
        assert pairs.numel() == 0
        n = len(seqs)
        seed[0] += 1
        qkv = wl.normal_tensor(seed[0], 3, (n, (h + 2 * hkv) * d), dtype=dtype).cuda()
        q = qkv[:, :h * d].view(n, h, d)
        k = qkv[:, h * d:(h + hkv) * d].view(n, hkv, d)
        v = qkv[:, (h + hkv) * d:].view(n, hkv, d)
        pos = torch.tensor([p for s in range(N) for p in positions[s]], dtype=torch.int32, device="cuda")
        out = torch.empty((n, h, d), dtype=dtype, device="cuda")
        pa.pa_rope_append_kv(out, q, k, v, pos, slots.cuda(), f, kc, vc, err_word=err)
        kr = pa.pa_rope(torch.empty_like(k.contiguous()), k, pos, f)
        for i, s in enumerate(seqs):
            for g in range(hkv):
                rows[s][g].append((kr[i, g].double(), v[i, g].double()))
        return out

    def attend_rows(q, s, index, scores=None):
        """q [h, d] over the listed rows of sequence s (None: all)."""
        out = torch.zeros((h, d), dtype=torch.float64, device="cuda")
        for g in range(hkv):
            at = rows[s][g] if index is None else [rows[s][g][i] for i in index]
            k, v = torch.stack([r[0] for r in at]), torch.stack([r[1] for r in at])
            G = h // hkv
            w = torch.softmax(q[g * G:(g + 1) * G].double() @ k.T / math.sqrt(d), -1)
            out[g * G:(g + 1) * G] = w @ v
            if scores is not None:
                scores[s][g] = scores[s][g] + w.sum(0)
        return out

    def close(got, want):
        # weights and output rounded to bf16: 2 x 2^-8 relative, on outputs of order one
        assert (got.double() - want).abs().max() <= 2 * 2 ** -8 * 4

    for s in range(N):
        bm.add_sequence(s)
    lens = [150, 37]
    tokens(lens, [list(range(150)), list(range(37))])
    # a drafted tree: two branches from the last committed token
    parents = torch.tensor([[-1, 0, 0, 1, 3], [-1, -1, 1, 2, 2]])
    depth = [[0, 1, 1, 2, 3], [0, 0, 1, 2, 2]]
    q = tokens([5, 5], [[lens[s] + x for x in depth[s]] for s in range(N)])
    tables, l5 = bm.tables()
    mask = pa.tree_mask_from_parents(parents)
    out = torch.empty((N, 5, h, d), dtype=dtype, device="cuda")
    pa.pa_decode_tree(out, q.view(N, 5, h, d), kc, vc, tables.cuda(), l5.cuda(), tree_mask=mask.cuda(), err_word=err)
    for s in range(N):
        for i in range(5):
            seen = list(range(lens[s])) + [lens[s] + j for j in range(5) if (int(mask[s, i, 0]) >> j) & 1]
            close(out[s, i], attend_rows(q[s * 5 + i], s, seen))
    # commit 0 -> 1 -> 3 of the first, 1 -> 2 of the second
    paths = [[0, 1, 3], [1, 2]]
    keep = torch.full((N, 1, 5), -1, dtype=torch.int32)
    for s, p in enumerate(paths):
        keep[s, 0, :len(p)] = torch.tensor(p, dtype=torch.int32)
    pa.pa_compact_kv(kc, vc, keep.cuda(), torch.tensor([3, 2], dtype=torch.int32).cuda(), tables.cuda(),
                     base_lens=torch.tensor(lens, dtype=torch.int32).cuda(), err_word=err)
    for s, p in enumerate(paths):
        for g in range(hkv):
            rows[s][g] = rows[s][g][:lens[s]] + [rows[s][g][lens[s] + j] for j in p]
        lens[s] += len(p)
        bm.truncate(s, lens[s])
    # two decode steps with scores
    sc = torch.zeros((N, hkv, M * bs), device="cuda")
    model = [[torch.zeros(1, dtype=torch.float64, device="cuda")[:0] for _ in range(hkv)] for _ in range(N)]
    position = list(lens)
    for _ in range(2):
        q = tokens([1, 1], [[position[0]], [position[1]]])
        position = [p + 1 for p in position]
        lens = [n + 1 for n in lens]
        tables, lt = bm.tables()
        for s in range(N):
            for g in range(hkv):
                pad = torch.zeros(lens[s] - model[s][g].numel(), dtype=torch.float64, device="cuda")
                model[s][g] = torch.cat([model[s][g], pad])
        o = torch.empty((N, h, d), device="cuda")
        pa.pa_decode_scored(o, sc, q, kc, vc, tables.cuda(), lt.cuda(), scores_in=sc, err_word=err)
        for s in range(N):
            close(o[s], attend_rows(q[s], s, None, model))
            for g in range(hkv):
                assert (sc[s, g, :lens[s]].double() - model[s][g]).abs().max() < 1e-4
    # evict to 64 tokens into renewed blocks (the second sequence is shorter)
    keep = torch.empty((N, hkv, 64), dtype=torch.int32, device="cuda")
    new = torch.empty(N, dtype=torch.int32, device="cuda")
    pa.pa_evict_select(keep, new, sc, sc, lt.cuda(), budget=64, recent=16, err_word=err)
    for s in range(N):
        bm.renew(s, min(lens[s], 64))
    dst, lt2 = bm.tables()
    pa.pa_compact_kv(kc, vc, keep, new, tables.cuda(), dst_block_tables=dst.cuda(), err_word=err)
    assert new.tolist() == [min(n, 64) for n in lens] == lt2.tolist()
    for s in range(N):
        for g in range(hkv):
            chosen = keep[s, g, :int(new[s])].tolist()
            assert chosen == sorted(set(chosen)) and chosen[-16:] == list(range(lens[s] - 16, lens[s]))
            assert (sc[s, g, :len(chosen)].double() - model[s][g][chosen]).abs().max() < 1e-4
            rows[s][g] = [rows[s][g][j] for j in chosen]
    lens = [min(n, 64) for n in lens]
    q = tokens([1, 1], [[position[0]], [position[1]]])
    tables, lt = bm.tables()
    o = torch.empty((N, h, d), device="cuda")
    pa.pa_decode(o, q, kc, vc, tables.cuda(), lt.cuda(), err_word=err)
    for s in range(N):
        close(o[s], attend_rows(q[s], s, None))
    assert err.item() == 0
