"""Operators of a paged KV-cache decode step, as cases to time and compare.

Four operators, each in its plain form (elementary torch operations, 32-bit
arithmetic, 64 bits where angles are formed) and as this package's calls:

  rope    rotate queries and keys by their positions, keys and values into
          their cache slots                            (pa_rope_append_kv)
  tree    attention of a tree of drafted tokens over the paged cache
                                                           (pa_decode_tree)
  scored  decode attention that adds each cached token's softmax weight to
          its accumulated score                          (pa_decode_scored)
  evict   keep the most recent and the highest-scored tokens of every kv head
          and move their rows into other blocks
                                        (pa_evict_select, pa_compact_kv)
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ELT = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one decode step of a handful of sequences on a small fp32 model: a launch's latency
        dict(name="rope_step_small", op="rope", tokens=4, heads=4, kv_heads=4, d=64, rot=64, interleaved=False,
             scaling="none", max_pos=100, block=16, dtype="f32"),
        # one decode step of a large batch with grouped heads, half of each head rotated, contexts stretched
        # eightfold by wavelength, far positions; q, k and v are slices of one fused projection
        dict(name="rope_step_batch", op="rope", tokens=256, heads=32, kv_heads=8, d=128, rot=64, interleaved=False,
             scaling="ramp", max_pos=1000000, block=16, dtype="bf16"),
        # a prompt chunk of one head per kv head, adjacent pairs, positions interpolated linearly
        dict(name="rope_prompt", op="rope", tokens=16384, heads=40, kv_heads=40, d=128, rot=128, interleaved=True,
             scaling="linear", max_pos=16384, block=16, dtype="f16"),
        # a few short fp32 sequences with five drafted tokens each
        dict(name="tree_small", op="tree", seqs=4, draft=5, heads=4, kv_heads=4, d=64, min_len=1, max_len=100,
             block=16, dtype="f32"),
        # one head per kv head, eight drafted tokens, contexts of 512 to 2048
        dict(name="tree_single_heads", op="tree", seqs=64, draft=8, heads=40, kv_heads=40, d=128, min_len=512,
             max_len=2048, block=16, dtype="f16"),
        # grouped heads, sixteen drafted tokens, ragged contexts up to 8192
        dict(name="tree_batch", op="tree", seqs=64, draft=16, heads=32, kv_heads=8, d=128, min_len=16, max_len=8192,
             block=16, dtype="bf16"),
        # a wide tree over a few very long contexts
        dict(name="tree_long", op="tree", seqs=4, draft=64, heads=32, kv_heads=8, d=128, min_len=65536,
             max_len=131072, block=16, dtype="bf16"),
        # scoring a few short sequences
        dict(name="scored_small", op="scored", seqs=5, heads=8, kv_heads=8, d=128, min_len=1, max_len=1000,
             block=16, dtype="f16"),
        # scoring a full batch of grouped heads
        dict(name="scored_batch", op="scored", seqs=256, heads=32, kv_heads=8, d=128, min_len=16, max_len=8192,
             block=16, dtype="bf16"),
        # short fp32 contexts cut to 32 tokens; some are below the budget already
        dict(name="evict_small", op="evict", seqs=4, kv_heads=4, d=64, min_len=1, max_len=100, budget=32, recent=8,
             block=16, dtype="f32"),
        # a batch cut to 2048 tokens a kv head
        dict(name="evict_batch", op="evict", seqs=64, kv_heads=8, d=128, min_len=2049, max_len=8192, budget=2048,
             recent=256, block=16, dtype="bf16"),
        # two very long contexts cut to an odd number of tokens
        dict(name="evict_long", op="evict", seqs=2, kv_heads=8, d=128, min_len=65537, max_len=131072, budget=16001,
             recent=1000, block=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "tree", "scored", "evict"])
    d = rng.choice([64, 128, 128])
    block = rng.choice([8, 16, 32])
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8, 16, 40])
        heads = kv * rng.choice([1, 2, 4, 8]) if kv <= 8 else kv
        dtype = rng.choice(["f32", "f16", "bf16"])
        most = (1 << 29) // ((heads + 2 * kv) * d * ELT[dtype])
        return dict(op=op, tokens=_log_int(rng, 1, min(32768, most)), heads=heads, kv_heads=kv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, d - 6, 2]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "ramp"]), max_pos=_log_int(rng, 64, 4000000),
                    block=block, dtype=dtype)
    if op == "evict":
        kv = rng.choice([1, 2, 4, 8, 16])
        seqs = _log_int(rng, 1, 64)
        dtype = rng.choice(["f32", "f16", "bf16"])
        rows = 1 << 20 if dtype == "f32" else 1 << 21
        max_len = _log_int(rng, 32, max(64, min(131072, rows // 2 // (seqs * kv))))
        budget = _log_int(rng, 1, max_len)
        return dict(op=op, seqs=seqs, kv_heads=kv, d=d, min_len=rng.choice([1, (max_len + 1) // 2]), max_len=max_len,
                    budget=budget, recent=rng.randint(0, budget), block=block, dtype=dtype)
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 8])
    # fp32 caches are of small models: shorter contexts and smaller trees
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    seqs = _log_int(rng, 1, 128)
    top = (2048 if dtype == "f32" else 131072) * 8 // kv
    max_len = _log_int(rng, 1, max(2, min(65536, top * 2 // seqs)))
    c = dict(op=op, seqs=seqs, heads=heads, kv_heads=kv, d=d, min_len=rng.choice([1, (max_len + 1) // 2]),
             max_len=max_len, block=block, dtype=dtype)
    if op == "tree":
        c["draft"] = _log_int(rng, 1, 12 if dtype == "f32" else 80)
    return c


# ---------------------------------------------------------------------------
# Inputs


def _lens(case):
    """Context lengths of a case, spread evenly over the logarithm of its range."""
    n, lo, hi = case["seqs"], case["min_len"], case["max_len"]
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _freqs(case, device):
    """Radians per position of each rotated pair, in 64 bits."""
    r = case["rot"]
    i = torch.arange(r // 2, dtype=torch.float64, device=device)
    base, factor, original = 10000.0, 8.0, 8192.0
    if case["scaling"] == "base" and r > 2:
        base = base * factor ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "ramp":
        turns = original * f / (2 * math.pi)  # rotations over the original context
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _tables(g, lens, block, extra=0):
    """Block tables over a shuffled pool that holds just what is needed: (tables, blocks in the pool)."""
    need = [(n + block - 1) // block for n in lens]
    width, total = max(max(need), 1), max(sum(need), 1) + extra
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    at = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    idx = (at[:, None] + j).clamp_max(total - 1)
    return torch.where(j < n[:, None], order[idx], torch.full_like(order[idx], -1)).contiguous(), total, order


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, d, bs = DT[case["dtype"]], case["d"], case["block"]
    st = dict(case=case)
    if case["op"] == "rope":
        T, H, K = case["tokens"], case["heads"], case["kv_heads"]
        qkv = _normal(g, (T, (H + 2 * K) * d), dt)
        st["q"] = qkv[:, :H * d].view(T, H, d)
        st["k"] = qkv[:, H * d:(H + K) * d].view(T, K, d)
        st["v"] = qkv[:, (H + K) * d:].view(T, K, d)
        st["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda").to(torch.int32)
        blocks = (T + bs - 1) // bs + 1
        slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:T]
        # a padded batch: about one row in sixteen has no slot
        pad = torch.rand(T, generator=g, device="cuda") < (1 / 16 if T > 8 else 0)
        st["slots"] = torch.where(pad, torch.full_like(slots, -1), slots).contiguous()
        st["freqs"] = _freqs(case, "cuda")
        st["mscale"] = 1.0 if case["scaling"] in ("none", "base") else 0.1 * math.log(8.0) + 1.0
        st["k_cache"] = _normal(g, (blocks, K, bs, d), dt)
        st["v_cache"] = _normal(g, (blocks, K, bs, d), dt)
        st["q_out"] = torch.empty((T, H, d), dtype=dt, device="cuda")
        return st
    lens = torch.tensor(_lens(case), device="cuda")
    lens = lens[torch.randperm(case["seqs"], generator=g, device="cuda")]
    N, K = case["seqs"], case["kv_heads"]
    if case["op"] == "evict":
        # a cached token's score is a sum of softmax weights: heavy-tailed, and exactly zero for some
        kept = [min(n, case["budget"]) for n in lens.tolist()]
        more = sum((n + bs - 1) // bs for n in kept)
        st["tables"], blocks, order = _tables(g, lens.tolist(), bs, extra=more)
        free = order[blocks - more:]
        n = (torch.tensor(kept, device="cuda") + bs - 1) // bs
        at, j = torch.cumsum(n, 0) - n, torch.arange(st["tables"].shape[1], device="cuda")
        st["dst_tables"] = torch.where(j < n[:, None], free[(at[:, None] + j).clamp_max(more - 1)],
                                       torch.full_like(free[:1], -1)).contiguous()
        width = st["tables"].shape[1] * bs
        s = torch.exp(1.5 * torch.randn((N, K, width), generator=g, device="cuda"))
        st["scores"] = torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.05, torch.zeros_like(s), s)
        st["scores_out"] = torch.empty_like(s)
        st["keep"] = torch.empty((N, K, case["budget"]), dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.empty(N, dtype=torch.int32, device="cuda")
        st["lens"] = lens.to(torch.int32)
    else:
        T = case["draft"] if case["op"] == "tree" else 0
        if T:
            # ragged trees: each node's parent is an earlier node, or the last committed token (-1)
            drafts = torch.randint((T + 1) // 2, T + 1, (N,), generator=g, device="cuda")
            parent = (torch.rand((N, T), generator=g, device="cuda") *
                      (torch.arange(T, device="cuda") + 1)).floor().long() - 1
            anc = torch.zeros((N, T, T + 1), dtype=torch.bool, device="cuda")
            rows = torch.arange(N, device="cuda")
            for i in range(T):
                if i:
                    up = parent[:, i]
                    anc[:, i] = anc[rows, up.clamp_min(0)] & (up >= 0)[:, None]
                anc[:, i, i] = True
            words = (T + 63) // 64
            bits = torch.zeros((N, T, words * 64), dtype=torch.int64, device="cuda")
            bits[:, :, :T] = anc[:, :, :T]
            one = torch.ones(64, dtype=torch.int64, device="cuda") << torch.arange(64, device="cuda")
            st["mask"] = (bits.view(N, T, words, 64) * one).sum(-1).contiguous()
            st["drafts"] = drafts.to(torch.int32)
            lens = lens + drafts
        st["lens"] = lens.to(torch.int32)
        st["tables"], blocks, _ = _tables(g, lens.tolist(), bs)
        shape = (N, T, case["heads"], d) if T else (N, case["heads"], d)
        st["q"] = _normal(g, shape, dt)
        st["out"] = torch.empty(shape, dtype=dt, device="cuda")
        if not T:
            width = st["tables"].shape[1] * bs
            s = torch.exp(1.5 * torch.randn((N, K, width), generator=g, device="cuda"))
            st["scores"] = s * (torch.arange(width, device="cuda") < lens[:, None, None])
            st["scores_out"] = torch.zeros_like(s)
    st["k_cache"] = _normal(g, (blocks, K, bs, d), dt)
    st["v_cache"] = _normal(g, (blocks, K, bs, d), dt)
    return st


# ---------------------------------------------------------------------------
# One pass


def run(st):
    case = st["case"]
    if own:
        return _OWN[case["op"]](st)
    return _PLAIN[case["op"]](st)


def _rotate(x, cos, sin, r, interleaved):
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y = x.float()
    xa, xb = y[..., a], y[..., b]
    ya, yb = xa * cos - xb * sin, xb * cos + xa * sin
    y = y.clone()
    y[..., a], y[..., b] = ya, yb
    return y.to(x.dtype)


def _plain_rope(st):
    case, bs = st["case"], st["case"]["block"]
    angle = st["positions"].double()[:, None] * st["freqs"]
    cos = (angle.cos() * st["mscale"]).float()[:, None]
    sin = (angle.sin() * st["mscale"]).float()[:, None]
    q = _rotate(st["q"], cos, sin, case["rot"], case["interleaved"])
    k = _rotate(st["k"], cos, sin, case["rot"], case["interleaved"])
    at = (st["slots"] >= 0).nonzero()[:, 0]
    slot = st["slots"][at]
    st["k_cache"][slot // bs, :, slot % bs] = k[at]
    st["v_cache"][slot // bs, :, slot % bs] = st["v"][at]
    return dict(q=q, k_cache=st["k_cache"], v_cache=st["v_cache"])


def _own_rope(st):
    from paged_kv_cache_251_gb300 import pa
    pa.pa_rope_append_kv(st["q_out"], st["q"], st["k"], st["v"], st["positions"], st["slots"], st["freqs"],
                         st["k_cache"], st["v_cache"], interleaved=st["case"]["interleaved"], mscale=st["mscale"])
    return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])


def _gather(cache, tables):
    """Every sequence's rows of a paged cache, [N, kv heads, table width * block, d], in 32 bits."""
    n, m = tables.shape
    x = cache[tables.clamp_min(0).long()]
    return x.permute(0, 2, 1, 3, 4).reshape(n, cache.shape[1], m * cache.shape[2], cache.shape[3]).float()


def _softmax(x, allowed):
    x = x.masked_fill(~allowed, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _plain_tree(st):
    case = st["case"]
    N, T, H, d = st["q"].shape
    K = case["kv_heads"]
    G = H // K
    k = _gather(st["k_cache"], st["tables"])
    L = k.shape[2]
    dev = k.device
    t = torch.arange(L, device=dev)
    lens, drafts = st["lens"].long(), st["drafts"].long()
    j = t[None, :] - (lens - drafts)[:, None]  # drafted index of each cached token, negative before
    inside = (j < drafts[:, None]) & (j >= 0)
    jc = j.clamp(0, T - 1)
    word = st["mask"].gather(2, (jc >> 6)[:, None, :].expand(N, T, L))
    bit = ((word >> (jc & 63)[:, None, :]) & 1).bool()
    allowed = (j < 0)[:, None, :] | (inside[:, None, :] & bit)
    allowed &= (torch.arange(T, device=dev)[None, :] < drafts[:, None])[:, :, None]
    q = st["q"].float().view(N, T, K, G, d).permute(0, 2, 1, 3, 4).reshape(N, K, T * G, d)
    x = (q @ k.transpose(2, 3)) * d ** -0.5
    del k
    p = _softmax(x.view(N, K, T, G, L), allowed[:, None, :, None, :]).view(N, K, T * G, L)
    o = p @ _gather(st["v_cache"], st["tables"])
    return o.view(N, K, T, G, d).permute(0, 2, 1, 3, 4).reshape(N, T, H, d).to(st["q"].dtype)


def _own_tree(st):
    from paged_kv_cache_251_gb300 import pa
    if "workspace" not in st:
        st["workspace"] = pa.tree_workspace_for(st["q"], st["k_cache"], st["tables"].shape[1])
    return pa.pa_decode_tree(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"],
                             tree_mask=st["mask"], draft_lens=st["drafts"], workspace=st["workspace"])


def _plain_scored(st):
    N, H, d = st["q"].shape
    K = st["case"]["kv_heads"]
    k = _gather(st["k_cache"], st["tables"])
    allowed = torch.arange(k.shape[2], device=k.device) < st["lens"].long()[:, None]
    x = (st["q"].float().view(N, K, H // K, d) @ k.transpose(2, 3)) * d ** -0.5
    p = _softmax(x, allowed[:, None, None, :])
    o = (p @ _gather(st["v_cache"], st["tables"])).view(N, H, d).to(st["q"].dtype)
    return dict(out=o, scores=st["scores"] + p.sum(2))


def _own_scored(st):
    from paged_kv_cache_251_gb300 import pa
    if "workspace" not in st:
        st["workspace"] = pa.scored_workspace_for(st["q"], st["k_cache"], st["tables"].shape[1])
    pa.pa_decode_scored(st["out"], st["scores_out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"],
                        scores_in=st["scores"], workspace=st["workspace"])
    return dict(out=st["out"], scores=st["scores_out"])


def _plain_evict(st):
    case, bs = st["case"], st["case"]["block"]
    N, K, W = st["scores"].shape
    B = case["budget"]
    dev = st["scores"].device
    t, lens = torch.arange(W, device=dev), st["lens"].long()
    valid = (t < lens[:, None])[:, None, :]
    recent = valid & (t >= (lens - case["recent"])[:, None])[:, None, :]
    key = torch.where(recent, torch.full_like(st["scores"], math.inf), st["scores"])
    key = torch.where(valid, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices  # ties: the lowest index first
    rank = torch.empty_like(order).scatter_(-1, order, t.expand(N, K, W))
    kept = valid & (rank < B)
    n = lens.clamp_max(B)
    place = torch.cumsum(kept, -1) - 1
    s, h, at = kept.nonzero(as_tuple=True)
    to = place[s, h, at]
    keep = torch.full((N, K, B), -1, dtype=torch.int32, device=dev)
    keep[s, h, to] = at.to(torch.int32)
    scores = torch.zeros_like(st["scores"])
    scores[s, h, to] = st["scores"][s, h, at]
    src, dst = st["tables"].long()[s, at // bs], st["dst_tables"].long()[s, to // bs]
    st["k_cache"][dst, h, to % bs] = st["k_cache"][src, h, at % bs]
    st["v_cache"][dst, h, to % bs] = st["v_cache"][src, h, at % bs]
    return dict(keep=keep, lens=n.to(torch.int32), scores=scores, k_cache=st["k_cache"], v_cache=st["v_cache"])


def _own_evict(st):
    from paged_kv_cache_251_gb300 import pa
    case = st["case"]
    pa.pa_evict_select(st["keep"], st["new_lens"], st["scores_out"], st["scores"], st["lens"], budget=case["budget"],
                       recent=case["recent"])
    pa.pa_compact_kv(st["k_cache"], st["v_cache"], st["keep"], st["new_lens"], st["tables"],
                     dst_block_tables=st["dst_tables"])
    return dict(keep=st["keep"], lens=st["new_lens"], scores=st["scores_out"], k_cache=st["k_cache"],
                v_cache=st["v_cache"])


_PLAIN = dict(rope=_plain_rope, tree=_plain_tree, scored=_plain_scored, evict=_plain_evict)
_OWN = dict(rope=_own_rope, tree=_own_tree, scored=_own_scored, evict=_own_evict)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    d, e = case["d"], ELT[case["dtype"]]
    if case["op"] == "rope":
        T, H, K = case["tokens"], case["heads"], case["kv_heads"]
        # q, k and v rows read and written once, positions and slots read
        return dict(bytes=2 * T * (H + 2 * K) * d * e + 12 * T + 4 * case["rot"], flops=3 * T * (H + K) * case["rot"])
    N, K, bs = case["seqs"], case["kv_heads"], case["block"]
    lens = _lens(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        width = (max(lens) + bs - 1) // bs * bs
        # every score read, the new row of scores and the kept list written, kept rows read and written
        return dict(bytes=4 * K * sum(lens) + 4 * N * K * (width + case["budget"]) + 4 * K * kept * d * e, flops=0)
    H, T = case["heads"], case.get("draft", 1)
    toks = sum(n + (3 * T + 1) // 4 for n in lens) if case["op"] == "tree" else sum(lens)
    b = toks * 2 * K * d * e + 2 * N * T * H * d * e + 4 * (toks // bs)
    if case["op"] == "tree":
        return dict(bytes=b + 8 * N * T * ((T + 63) // 64), flops=4 * toks * ((3 * T + 1) // 4) * H * d)
    return dict(bytes=b + 8 * K * toks, flops=4 * toks * H * d)


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return dict(rope=_exact_rope, tree=_exact_tree, scored=_exact_scored, evict=_exact_evict)[case["op"]](st)


def _exact_rope(st):
    case, r = st["case"], st["case"]["rot"]
    pairs = [(2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2) for i in range(r // 2)]
    turn = torch.polar(torch.full((), st["mscale"], dtype=torch.float64, device="cuda"),
                       st["positions"].double()[:, None] * st["freqs"][None, :])
    first, second = [a for a, _ in pairs], [b for _, b in pairs]

    def rotated(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k, v = st["k_cache"].double(), st["v_cache"].double()
    nb, K, bs, d = k.shape
    good = st["slots"] >= 0
    for cache, rows in ((k, rotated(st["k"])), (v, st["v"].double())):
        flat = cache.transpose(1, 2).reshape(nb * bs, K, d)
        flat[st["slots"][good]] = rows[good]
        cache.copy_(flat.view(nb, bs, K, d).transpose(1, 2))
    return dict(q=rotated(st["q"]), k_cache=k, v_cache=v)


def _rows_of(cache, table, n):
    """The first n cached rows of one sequence, [n, kv heads, d], in 64 bits."""
    bs = cache.shape[2]
    blocks = table[:(n + bs - 1) // bs].long()
    return cache[blocks].transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[:n].double()


def _exact_tree(st):
    N, T, H, d = st["q"].shape
    K = st["case"]["kv_heads"]
    out = torch.zeros((N, T, H, d), dtype=torch.float64, device="cuda")
    masks = st["mask"].tolist()
    for s, (n, drafted) in enumerate(zip(st["lens"].tolist(), st["drafts"].tolist())):
        k, v = _rows_of(st["k_cache"], st["tables"][s], n), _rows_of(st["v_cache"], st["tables"][s], n)
        q = st["q"][s, :drafted].double().view(drafted, K, H // K, d)
        bias = torch.zeros((drafted, n), dtype=torch.float64)
        for i in range(drafted):
            seen = [(masks[s][i][j // 64] >> (j % 64)) & 1 for j in range(drafted)]
            bias[i, n - drafted:] = torch.tensor([0.0 if b else -math.inf for b in seen], dtype=torch.float64)
        x = torch.einsum("ikgd,nkd->kgin", q, k) / math.sqrt(d) + bias.cuda()
        out[s, :drafted] = torch.einsum("kgin,nkd->ikgd", x.softmax(-1), v).reshape(drafted, H, d)
    return out


def _exact_scored(st):
    N, H, d = st["q"].shape
    K = st["case"]["kv_heads"]
    out = torch.zeros((N, H, d), dtype=torch.float64, device="cuda")
    scores = st["scores"].double().clone()
    for s, n in enumerate(st["lens"].tolist()):
        k, v = _rows_of(st["k_cache"], st["tables"][s], n), _rows_of(st["v_cache"], st["tables"][s], n)
        w = (torch.einsum("kgd,nkd->kgn", st["q"][s].double().view(K, H // K, d), k) / math.sqrt(d)).softmax(-1)
        out[s] = torch.einsum("kgn,nkd->kgd", w, v).reshape(H, d)
        scores[s, :, :n] += w.sum(1)
    return dict(out=out, scores=scores)


def _exact_evict(st):
    case, bs = st["case"], st["case"]["block"]
    keep = torch.full(st["keep"].shape, -1, dtype=torch.int32)
    scores = torch.zeros(st["scores"].shape, dtype=torch.float64)
    given = st["scores"].double().cpu()
    lens = st["lens"].tolist()
    k, v = st["k_cache"].double(), st["v_cache"].double()
    new = []
    for s, n in enumerate(lens):
        new.append(min(n, case["budget"]))
        late = range(max(0, n - case["recent"]), n)
        for h in range(case["kv_heads"]):
            row = given[s, h].tolist()
            early = sorted(range(len(range(0, late.start))), key=lambda t: (-row[t], t))
            chosen = sorted(early[:max(0, new[s] - len(late))] + list(late)[-new[s]:])
            keep[s, h, :new[s]] = torch.tensor(chosen, dtype=torch.int32)
            scores[s, h, :new[s]] = given[s, h, chosen]
            src = torch.tensor(chosen, device="cuda")
            dst = torch.arange(new[s], device="cuda")
            a, b = st["tables"][s][src // bs].long(), st["dst_tables"][s][dst // bs].long()
            k[b, h, dst % bs], v[b, h, dst % bs] = k[a, h, src % bs], v[a, h, src % bs]
    return dict(keep=keep, lens=torch.tensor(new, dtype=torch.int32), scores=scores, k_cache=k, v_cache=v)
