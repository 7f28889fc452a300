"""Operators of a speculative serving step over block-scaled 8-bit caches, as cases to time and compare.

Five operators, each in its plain form (elementary torch operations, 32-bit
arithmetic, 64 bits where a drawn token hangs on a sum) and as this package's
calls:

  verify   accept or reject drafted tokens (a chain or a tree) against the
           target's probabilities, and draw the token after them
                                                        (pa_verify_drafts)
  append   store new K/V rows in 8-bit blocks with one scale a block and head,
           the block's older rows re-coded when the scale grows
                                                (pa_append_kv_block_quant)
  decode   decode attention over such a cache      (pa_decode_block_quant)
  update   the block tables and reference counts of the next step: rows kept,
           forked, cut, freed and grown, shared last blocks copied
                                          (pa_pages_update, pa_copy_pages)
  compact  the used blocks of a pool moved to its front
                                         (pa_pages_compact, pa_copy_pages)
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ELT = {"f32": 4, "f16": 2, "bf16": 2}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
QMAX = {"int8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one sequence with four drafted tokens in a chain: a call's latency
        dict(name="verify_small", op="verify", seqs=1, draft=4, vocab=32000, tree=False, with_q=True, dtype="f32"),
        # a batch of chains over a large vocabulary
        dict(name="verify_batch", op="verify", seqs=64, draft=7, vocab=128000, tree=False, with_q=True, dtype="f32"),
        # trees of drafted tokens over a vocabulary of odd size, 16-bit probabilities
        dict(name="verify_tree", op="verify", seqs=32, draft=24, vocab=50257, tree=True, with_q=True, dtype="bf16"),
        # the new token of each sequence of a decode step
        dict(name="append_step", op="append", seqs=64, min_len=1, max_len=1, kv_heads=8, d=128, block=16, code="int8",
             dtype="bf16"),
        # a chunk of ragged prompts
        dict(name="append_prompt", op="append", seqs=24, min_len=64, max_len=4096, kv_heads=8, d=128, block=16,
             code="e4m3", dtype="bf16"),
        # a few short sequences of a small fp32 model
        dict(name="decode_small", op="decode", seqs=4, heads=4, kv_heads=4, d=64, min_len=1, max_len=100, window=0,
             block=16, code="int8", dtype="f32"),
        # a full batch of grouped heads, ragged contexts
        dict(name="decode_batch", op="decode", seqs=256, heads=32, kv_heads=8, d=128, min_len=16, max_len=8192,
             window=0, block=16, code="int8", dtype="bf16"),
        # a few very long contexts
        dict(name="decode_long", op="decode", seqs=4, heads=32, kv_heads=8, d=128, min_len=65536, max_len=131072,
             window=0, block=32, code="e4m3", dtype="f16"),
        # every sequence of a batch keeps most of its drafted tokens and reserves room for four more; a few have
        # ended and their rows start anew
        dict(name="update_step", op="update", rows=256, beams=1, min_len=16, max_len=8192, cut=3, grow=4, block=16,
             kv_heads=2, d=64, spare=1024, dtype="bf16"),
        # a step of beam search: 32 prompts of 2000 tokens, 8 beams each, forked from the best ones
        dict(name="update_beams", op="update", rows=256, beams=8, min_len=1850, max_len=2250, cut=0, grow=1, block=16,
             kv_heads=8, d=128, spare=1024, dtype="f16"),
        # a small pool, a third in use
        dict(name="compact_small", op="compact", rows=16, min_len=1, max_len=1000, block=16, kv_heads=4, d=64,
             blocks=1024, dtype="f32"),
        # a large pool in use by two thirds, its used blocks scattered
        dict(name="compact_large", op="compact", rows=256, min_len=16, max_len=8192, block=16, kv_heads=4, d=128,
             blocks=38000, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "append", "decode", "decode", "update", "compact"])
    if op == "verify":
        tree = rng.random() < 0.5
        vocab = _log_int(rng, 500, 150000)
        draft = _log_int(rng, 1, 48 if tree else 16)
        most = (1 << 26) // (vocab * (draft + 1))
        return dict(op=op, seqs=_log_int(rng, 1, max(1, min(256, most))), draft=draft, vocab=vocab, tree=tree,
                    with_q=rng.random() < 0.7, dtype=rng.choice(["f32", "f32", "f16", "bf16"]))
    d = rng.choice([64, 128, 128])
    block = rng.choice([8, 16, 32])
    if op == "append":
        kv = rng.choice([1, 2, 4, 8, 16, 40])
        most = max(1, (1 << 24) // (kv * d))
        if rng.random() < 0.5:
            seqs, lo, hi = _log_int(rng, 1, min(512, most)), 1, 1
        else:
            hi = _log_int(rng, 2, min(8192, most))
            seqs, lo = _log_int(rng, 1, max(1, min(64, most // hi))), max(1, hi // 16)
        return dict(op=op, seqs=seqs, min_len=lo, max_len=hi, kv_heads=kv, d=d, block=block,
                    code=rng.choice(["int8", "e4m3"]), dtype=rng.choice(["f32", "f16", "bf16"]))
    if op == "decode":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 8])
        seqs = _log_int(rng, 1, 256)
        max_len = _log_int(rng, 1, max(2, min(131072, (1 << 19) * 8 // (kv * seqs))))
        return dict(op=op, seqs=seqs, heads=heads, kv_heads=kv, d=d, min_len=rng.choice([1, (max_len + 1) // 2]),
                    max_len=max_len, window=rng.choice([0, 0, 0, _log_int(rng, 1, max_len + 1)]), block=block,
                    code=rng.choice(["int8", "e4m3"]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    kv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "update":
        beams = rng.choice([1, 1, 2, 4, 7])
        rows = beams * _log_int(rng, 1, 300 // beams)
        max_len = _log_int(rng, 4, min(8192, (1 << 27) // (rows * kv * d * 2)))
        return dict(op=op, rows=rows, beams=beams, min_len=max(1, max_len // rng.choice([1, 2, 64])), max_len=max_len,
                    cut=rng.choice([0, 1, 5]), grow=rng.choice([1, 1, 4, 17, 100]), block=block, kv_heads=kv, d=d,
                    spare=_log_int(rng, 1, 4000), dtype=dtype)
    rows = _log_int(rng, 1, 256)
    max_len = _log_int(rng, 1, min(8192, (1 << 27) // (rows * kv * d * 2)))
    need = rows * ((max_len + block - 1) // block)
    return dict(op=op, rows=rows, min_len=max(1, max_len // 16), max_len=max_len, block=block, kv_heads=kv, d=d,
                blocks=need + _log_int(rng, 1, max(2, need)), dtype=dtype)


# ---------------------------------------------------------------------------
# Inputs


def _lens(n, lo, hi):
    """n lengths spread evenly over the logarithm of [lo, hi]."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _up(x, block):
    return (x + block - 1) // block


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _gumbel(g, shape):
    return -torch.log(-torch.log(torch.rand(shape, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))


def _tables(need, width, order):
    """Tables [len(need), width] of the ids in `order`, handed out row by row; -1 past each row's need."""
    at = torch.cumsum(need, 0) - need
    j = torch.arange(width, device="cuda")
    ids = order[(at[:, None] + j).clamp_max(order.numel() - 1)]
    return torch.where(j < need[:, None], ids, torch.full_like(ids, -1)).to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = dict(case=case)
    dict(verify=_prepare_verify, append=_prepare_append, decode=_prepare_decode, update=_prepare_update,
         compact=_prepare_compact)[case["op"]](st, case, g)
    return st


def _prepare_verify(st, case, g):
    N, T, V, dt = case["seqs"], case["draft"], case["vocab"], DT[case["dtype"]]
    # logits of which a few dominate; the draft model is near the target
    target = 3 * _normal(g, (N, T + 1, V), torch.float32)
    st["draft_probs"] = None
    if case["with_q"]:
        draft = target[:, :T] + 0.8 * _normal(g, (N, T, V), torch.float32)
        st["draft_probs"] = draft.softmax(-1).to(dt)
    else:
        draft = target[:, :T]
    i = torch.arange(T, device="cuda")
    if case["tree"]:
        # a node's parent is one of the four nodes before it, or the last committed token
        back = torch.randint(1, 5, (N, T), generator=g, device="cuda")
        st["parents"] = (i - back).clamp_min(-1).to(torch.int32)
        at = st["parents"].long() + 1
    else:
        st["parents"] = None
        at = i.expand(N, T)
    # each drafted token is drawn from the draft's distribution behind its parent
    tokens = torch.empty((N, T), dtype=torch.int64, device="cuda")
    rows = torch.arange(N, device="cuda")
    for k in range(T):
        tokens[:, k] = (draft[rows, at[:, k]] + _gumbel(g, (N, V))).argmax(-1)
    st["draft_tokens"] = tokens.to(torch.int32)
    st["target_probs"] = target.softmax(-1).to(dt)
    st["draft_lens"] = torch.randint((T + 1) // 2, T + 1, (N,), generator=g, device="cuda").to(torch.int32)
    st["uniforms"] = torch.rand((N, T + 1), generator=g, device="cuda")
    st["accept_lens"] = torch.empty(N, dtype=torch.int32, device="cuda")
    st["accepted"] = torch.empty((N, T), dtype=torch.int32, device="cuda")
    st["tokens"] = torch.empty((N, T + 1), dtype=torch.int32, device="cuda")


def _codes(g, shape, code):
    """Codes as a block's absolute maximum leaves them: normal values, the largest of about 3.5 at the code's limit."""
    out = torch.empty(shape, dtype=CODE[code], device="cuda")
    for part in out.split(max(1, (1 << 27) // max(1, out[0].numel()))):
        x = _normal(g, part.shape, torch.float32).mul_(QMAX[code] / 3.5).clamp_(-QMAX[code], QMAX[code])
        part.copy_(x.round_() if code == "int8" else x)
    return out


def _prepare_append(st, case, g):
    K, d, bs, dt = case["kv_heads"], case["d"], case["block"], DT[case["dtype"]]
    lens = torch.tensor(_lens(case["seqs"], case["min_len"], case["max_len"]), device="cuda")
    # where each sequence stands: a single token anywhere, a prompt mostly at a block's start
    start = torch.randint(0, bs, lens.shape, generator=g, device="cuda")
    if case["max_len"] > 1:
        start = torch.where(torch.rand(lens.shape, generator=g, device="cuda") < 0.75, torch.zeros_like(start), start)
    need = (start + lens + bs - 1) // bs
    nb = sum(_up(n + bs - 1, bs) for n in lens.tolist()) + 2
    order = torch.randperm(nb, generator=g, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens)
    T = seq.numel()
    t = torch.arange(T, device="cuda") - (torch.cumsum(lens, 0) - lens)[seq] + start[seq]
    st["slots"] = order[(torch.cumsum(need, 0) - need)[seq] + t // bs] * bs + t % bs
    if T > 8:  # a padded batch
        pad = torch.rand(T, generator=g, device="cuda") < 1 / 16
        st["slots"] = torch.where(pad, torch.full_like(st["slots"], -1), st["slots"]).contiguous()
    # rows of differing size, so that some enlarge their block's scale
    size = torch.exp(0.5 * torch.randn((T, K, 1), generator=g, device="cuda"))
    st["k"] = (_normal(g, (T, K, d), torch.float32) * size).to(dt)
    st["v"] = (_normal(g, (T, K, d), torch.float32) * size).to(dt)
    for name in ("k", "v"):
        st[name + "_cache"] = _codes(g, (nb, K, bs, d), case["code"])
        st[name + "_scales"] = (torch.rand((nb, K), generator=g, device="cuda") + 0.5) * (4 / QMAX[case["code"]])


def _prepare_decode(st, case, g):
    N, H, K, d, bs = case["seqs"], case["heads"], case["kv_heads"], case["d"], case["block"]
    lens = torch.tensor(_lens(N, case["min_len"], case["max_len"]), device="cuda")
    lens = lens[torch.randperm(N, generator=g, device="cuda")]
    need = (lens + bs - 1) // bs
    nb = int(need.sum()) + 3
    order = torch.randperm(nb, generator=g, device="cuda")
    st["tables"] = _tables(need, int(need.max()), order)
    st["lens"] = lens.to(torch.int32)
    st["q"] = _normal(g, (N, H, d), DT[case["dtype"]])
    st["out"] = torch.empty_like(st["q"])
    for name in ("k", "v"):
        st[name + "_cache"] = _codes(g, (nb, K, bs, d), case["code"])
        st[name + "_scales"] = (torch.rand((nb, K), generator=g, device="cuda") + 0.5) * (3.5 / QMAX[case["code"]])


def _pools(st, case, g, nb):
    shape = (nb, case["kv_heads"], case["block"], case["d"])
    st["k_cache"], st["v_cache"] = (_normal(g, shape, DT[case["dtype"]]) for _ in range(2))


def _prepare_update(st, case, g):
    N, B, bs = case["rows"], case["beams"], case["block"]
    lens = torch.tensor(_lens(N // B, case["min_len"], case["max_len"]), device="cuda")
    lens = lens[torch.randperm(N // B, generator=g, device="cuda")].repeat_interleave(B)
    row = torch.arange(N, device="cuda")
    have = (lens + bs - 1) // bs
    # the beams of a prompt share the whole blocks of its first nine tenths
    shared = (lens * 9 // 10) // bs if B > 1 else torch.zeros_like(lens)
    if B > 1:
        parents = row // B * B + torch.randint(0, B, (N,), generator=g, device="cuda")
    else:
        ended = torch.randperm(N, generator=g, device="cuda") < N // 20
        parents = torch.where(ended, torch.full_like(row, -1), row)
    keep = (lens - torch.randint(0, case["cut"] + 1, (N,), generator=g, device="cuda")).clamp_min(0)
    grow = keep + case["grow"]
    if B == 1:
        fresh = torch.randint(1, case["max_len"] + 1, (N,), generator=g, device="cuda") // 4 + 1
        keep, grow = torch.where(ended, 0, keep), torch.where(ended, fresh, grow)
    width = _up(case["max_len"] + case["grow"], bs)
    taken = have - torch.where(row % B == 0, 0, shared)
    used = int(taken.sum())
    new_rows = N // 20 * _up(case["max_len"] // 4 + 1, bs) if B == 1 else 0
    nb = used + N * (2 + _up(case["grow"], bs)) + new_rows + case["spare"]
    order = torch.randperm(nb, generator=g, device="cuda")
    mine = _tables(taken, width, order)
    j = torch.arange(width, device="cuda")
    first = row // B * B
    lead = mine[first]
    back = (j - torch.where(row % B == 0, 0, shared)[:, None]).clamp_min(0)
    tables = torch.where(j < shared[:, None], lead, mine.gather(1, back))
    st["tables"] = torch.where(j < have[:, None], tables, torch.full_like(tables, -1)).contiguous()
    held = st["tables"][st["tables"] >= 0].long()
    st["refs"] = torch.bincount(held, minlength=nb).to(torch.int32)
    for name, x in (("lens", lens), ("parents", parents), ("keep", keep), ("grow", grow)):
        st[name] = x.to(torch.int32)
    st["new_tables"], st["new_refs"] = torch.empty_like(st["tables"]), torch.empty_like(st["refs"])
    st["pairs"] = torch.empty((N, 2), dtype=torch.int64, device="cuda")
    st["status"] = torch.empty(4, dtype=torch.int32, device="cuda")
    _pools(st, case, g, nb)


def _prepare_compact(st, case, g):
    N, bs, nb = case["rows"], case["block"], case["blocks"]
    lens = torch.tensor(_lens(N, case["min_len"], case["max_len"]), device="cuda")
    lens = lens[torch.randperm(N, generator=g, device="cuda")]
    need = (lens + bs - 1) // bs
    order = torch.randperm(nb, generator=g, device="cuda")
    st["tables"] = _tables(need, int(need.max()), order)
    # some blocks are held by a prompt cache too
    more = (torch.rand(nb, generator=g, device="cuda") < 0.1).to(torch.int32)
    used = torch.zeros(nb, dtype=torch.int32, device="cuda")
    used[st["tables"][st["tables"] >= 0].long()] = 1
    st["refs"] = used * (1 + more)
    st["lens"] = lens.to(torch.int32)
    st["new_tables"], st["new_refs"] = torch.empty_like(st["tables"]), torch.empty_like(st["refs"])
    st["remap"] = torch.empty_like(st["refs"])
    st["pairs"] = torch.empty((nb // 2, 2), dtype=torch.int64, device="cuda")
    st["status"] = torch.empty(4, dtype=torch.int32, device="cuda")
    _pools(st, case, g, nb)


# ---------------------------------------------------------------------------
# One pass


def run(st):
    case = st["case"]
    if own:
        return _OWN[case["op"]](st)
    return _PLAIN[case["op"]](st)


def _plain_verify(st):
    P, Q, tok, u = st["target_probs"], st["draft_probs"], st["draft_tokens"].long(), st["uniforms"].double()
    N, T = tok.shape
    V, dev = P.shape[2], P.device
    row, i = torch.arange(N, device=dev), torch.arange(T, device=dev)
    parent = i.expand(N, T) - 1 if st["parents"] is None else st["parents"].long()
    node = torch.full((N,), -1, dtype=torch.int64, device=dev)
    # the weights of a node's next token: max(0, p - a q), S in all (a = 0, S = 1 before any rejection); without
    # draft probabilities p without the tokens in `gone`
    a, S = torch.zeros(N, dtype=torch.float64, device=dev), torch.ones(N, dtype=torch.float64, device=dev)
    gone = torch.zeros((N, V), dtype=torch.bool, device=dev) if Q is None else None
    taken = torch.zeros((N, T), dtype=torch.bool, device=dev)
    for k in range(T):  # a token's fate hangs on those before it
        here = (parent[:, k] == node) & (k < st["draft_lens"])
        x = tok[:, k]
        p = P[row, node + 1, x].double()
        if Q is None:
            p = torch.where(gone[row, x], torch.zeros_like(p), p)
            ok = here & (u[:, k] * S < p)
            lost = here & ~ok
            S = torch.where(ok, torch.ones_like(S), torch.where(lost, S - p, S))
            gone[row, x] |= lost
            gone &= ~ok[:, None]
        else:
            at = (node + 1).clamp_max(T - 1)
            q = Q[row, at, x].double()
            ok = here & (u[:, k] * S * q < (p - a * q).clamp_min(0))
            lost = here & ~ok
            a = torch.where(ok, torch.zeros_like(a), torch.where(lost, a + S, a))
            total = (P[row, node + 1].double() - a[:, None] * Q[row, at].double()).clamp_min_(0).sum(-1)
            S = torch.where(ok, torch.ones_like(S), torch.where(lost, total, S))
        taken[:, k] = ok
        node = torch.where(ok, torch.full_like(node, k), node)
    p = P[row, node + 1].double()
    if Q is None:
        w = torch.where(gone, torch.zeros_like(p), p)
    else:
        w = (p - a[:, None] * Q[row, (node + 1).clamp_max(T - 1)].double()).clamp_min_(0)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
    cum = w.cumsum(-1)
    total = cum[:, -1:]
    last = (w > 0).to(torch.int64).mul_(torch.arange(1, V + 1, device=dev)).amax(-1) - 1
    x = torch.minimum((cum <= u[:, T:] * total).sum(-1), last)
    n = taken.sum(-1)
    order = torch.sort((~taken).to(torch.int32), dim=-1, stable=True).indices
    accepted = torch.where(i < n[:, None], order, torch.full_like(order, -1))
    tokens = torch.where(i < n[:, None], tok.gather(1, order), torch.full_like(order, -1))
    tokens = torch.cat([tokens, torch.full_like(tokens[:, :1], -1)], 1).scatter(1, n[:, None], x[:, None])
    return dict(accept_lens=n.to(torch.int32), accepted=accepted.to(torch.int32), tokens=tokens.to(torch.int32))


def _own_verify(st):
    from paged_kv_cache_251_gb300 import pa
    pa.pa_verify_drafts(st["accept_lens"], st["accepted"], st["tokens"], st["target_probs"], st["draft_tokens"],
                        st["uniforms"], draft_probs=st["draft_probs"], draft_lens=st["draft_lens"],
                        parents=st["parents"])
    return dict(accept_lens=st["accept_lens"], accepted=st["accepted"], tokens=st["tokens"])


def _encode(x, code):
    if code == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _values(st):
    """The cache after a pass: E4M3 codes are values as they stand (of their block's scale), integers are scaled."""
    out = {}
    for name in ("k", "v"):
        c, s = st[name + "_cache"], st[name + "_scales"]
        out[name + "_cache"] = c if st["case"]["code"] == "e4m3" else c * s[:, :, None, None]
        out[name + "_scales"] = s
    return out


def _plain_append(st):
    case, bs, code = st["case"], st["case"]["block"], st["case"]["code"]
    at = (st["slots"] >= 0).nonzero()[:, 0]
    slot = st["slots"][at]
    block, off = slot // bs, slot % bs
    for name in ("k", "v"):
        x, cache, scales = st[name][at].float(), st[name + "_cache"], st[name + "_scales"]
        nb, K = scales.shape
        amax = torch.zeros((nb, K), device=x.device)
        amax.scatter_reduce_(0, block[:, None].expand(-1, K), x.abs().amax(-1), "amax")
        written = torch.zeros((nb, bs), dtype=torch.bool, device=x.device)
        written[block, off] = True
        touched, fresh = written.any(1), written[:, 0]
        mine = amax / torch.full_like(amax, QMAX[code])
        scale = torch.where(fresh[:, None], mine, torch.maximum(mine, scales))
        scale = torch.where(touched[:, None], scale, scales)
        # a scale that grew: the rows of before are coded anew
        grew = (touched & ~fresh)[:, None] & (scale > scales)
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        b, h = grew.nonzero(as_tuple=True)
        cache[b, h] = _encode(cache[b, h].float() * scales[b, h][:, None, None] / safe[b, h][:, None, None], code)
        y = torch.where(scale[block][:, :, None] > 0, x / safe[block][:, :, None], torch.zeros_like(x))
        cache[block, :, off] = _encode(y, code)
        scales.copy_(scale)
    return _values(st)


def _own_append(st):
    from paged_kv_cache_251_gb300 import pa
    if "workspace" not in st:
        st["workspace"] = pa.append_block_quant_workspace_for(st["slots"], st["k_cache"])
    pa.pa_append_kv_block_quant(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["k_scales"],
                                st["v_scales"], workspace=st["workspace"])
    return _values(st)


def _gather(cache, scales, tables):
    """Every sequence's rows of a block-scaled cache, [N, kv heads, table width * block, d], in 32 bits."""
    n, m = tables.shape
    t = tables.clamp_min(0).long()
    x = cache[t].float().mul_(scales[t][:, :, :, None, None])
    return x.permute(0, 2, 1, 3, 4).reshape(n, cache.shape[1], m * cache.shape[2], cache.shape[3])


def _softmax(x, allowed):
    x = x.masked_fill(~allowed, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _plain_decode(st):
    N, H, d = st["q"].shape
    K, window = st["case"]["kv_heads"], st["case"]["window"]
    k = _gather(st["k_cache"], st["k_scales"], st["tables"])
    t, lens = torch.arange(k.shape[2], device=k.device), st["lens"].long()
    allowed = t < lens[:, None]
    if window:
        allowed &= t >= (lens - window)[:, None]
    x = (st["q"].float().view(N, K, H // K, d) @ k.transpose(2, 3)) * d ** -0.5
    del k
    p = _softmax(x, allowed[:, None, None, :])
    o = p @ _gather(st["v_cache"], st["v_scales"], st["tables"])
    return o.view(N, H, d).to(st["q"].dtype)


def _own_decode(st):
    from paged_kv_cache_251_gb300 import pa
    if "workspace" not in st:
        st["workspace"] = pa.block_quant_workspace_for(st["q"], st["k_cache"], st["tables"].shape[1])
    return pa.pa_decode_block_quant(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                                    st["tables"], st["lens"], window=st["case"]["window"],
                                    workspace=st["workspace"])


def _plain_copy(st, pairs):
    src, dst = pairs[pairs[:, 0] >= 0].unbind(1)
    for name in ("k_cache", "v_cache"):
        st[name][dst] = st[name][src]


def _plain_update(st):
    bs, tables, lens = st["case"]["block"], st["tables"].long(), st["lens"].long()
    N, M = tables.shape
    nb, dev = st["refs"].numel(), tables.device
    row, j = torch.arange(N, device=dev), torch.arange(M, device=dev)
    parent = st["parents"].long()
    src = tables[parent.clamp_min(0)]
    keep = torch.where(parent >= 0, torch.minimum(st["keep"].long(), lens[parent.clamp_min(0)]), 0).clamp_min(0)
    grow = torch.maximum(st["grow"].long(), keep).clamp_max(M * bs)
    kept, total = (keep + bs - 1) // bs, (grow + bs - 1) // bs
    # references after the rows of before let go and the new ones hold what they keep
    refs = st["refs"].long() - torch.bincount(tables[j < ((lens + bs - 1) // bs)[:, None]], minlength=nb)
    refs = refs + torch.bincount(src[j < kept[:, None]], minlength=nb)
    # a last block that is written to stays if all who hold it write to it, and then with the lowest row
    writes = (grow > keep) & (keep % bs != 0)
    last = src.gather(1, (kept - 1).clamp_min(0)[:, None])[:, 0].clamp_min(0)
    writers = torch.bincount(last, weights=writes.double(), minlength=nb).long()
    lowest = torch.full((nb,), N, device=dev).scatter_reduce_(0, last, torch.where(writes, row, N), "amin")
    copied = writes & ~((writers[last] == refs[last]) & (lowest[last] == row))
    need = total - kept + copied
    free = torch.sort((refs != 0).to(torch.int32), stable=True).indices
    at, spare = torch.cumsum(need, 0) - need, (refs == 0).sum()
    done = need.sum() <= spare
    place = at[:, None] + copied[:, None] + (j - kept[:, None])
    new = torch.where(j < kept[:, None], src, torch.full_like(src, -1))
    new = torch.where((j >= kept[:, None]) & (j < total[:, None]), free[place.clamp(0, nb - 1)], new)
    to = free[at.clamp_max(nb - 1)]
    new = torch.where((j == kept[:, None] - 1) & copied[:, None], to[:, None], new)
    pairs = torch.where((copied & done)[:, None], torch.stack([last, to], 1), torch.full((N, 2), -1, device=dev))
    refs = refs - torch.bincount(last, weights=copied.double(), minlength=nb).long()
    refs = refs + torch.bincount(new[(j >= kept[:, None]) & (j < total[:, None])], minlength=nb)
    refs = refs + torch.bincount(to, weights=copied.double(), minlength=nb).long()
    _plain_copy(st, pairs)
    status = torch.stack([done.long(), need.sum(), spare - need.sum() * done, (copied & done).sum()])
    return dict(tables=torch.where(done, new.to(torch.int32), st["new_tables"]),
                refs=torch.where(done, refs.to(torch.int32), st["new_refs"]), pairs=pairs,
                status=status.to(torch.int32), k_cache=st["k_cache"], v_cache=st["v_cache"])


def _own_update(st):
    from paged_kv_cache_251_gb300 import pa
    if "workspace" not in st:
        st["workspace"] = pa.pages_workspace_for(st["tables"], st["refs"])
    pa.pa_pages_update(st["new_tables"], st["new_refs"], st["pairs"], st["status"], st["tables"], st["refs"],
                       st["lens"], st["keep"], st["grow"], block_size=st["case"]["block"], parents=st["parents"],
                       workspace=st["workspace"])
    pa.pa_copy_pages(st["pairs"], [st["k_cache"], st["v_cache"]])
    return dict(tables=st["new_tables"], refs=st["new_refs"], pairs=st["pairs"], status=st["status"],
                k_cache=st["k_cache"], v_cache=st["v_cache"])


def _plain_compact(st):
    bs, refs = st["case"]["block"], st["refs"]
    nb, dev = refs.numel(), refs.device
    b = torch.arange(nb, device=dev)
    used = refs > 0
    U = used.sum()
    # the highest used block goes to the lowest free one, and so on, while it lies behind the front
    high, low = used & (b >= U), ~used & (b < U)
    moves = high.sum()
    src = torch.sort(torch.where(high, b, torch.full_like(b, -1)), descending=True).values
    dst = torch.sort(torch.where(low, b, torch.full_like(b, nb))).values
    k = torch.arange(st["pairs"].shape[0], device=dev)
    m = min(nb, k.numel())
    pairs = torch.full((k.numel(), 2), -1, dtype=torch.int64, device=dev)
    pairs[:m] = torch.where((k[:m] < moves)[:, None], torch.stack([src[:m], dst[:m]], 1), pairs[:m])
    go = pairs[:, 0] >= 0
    remap, new_refs = b.clone(), refs.clone()
    src, dst = pairs[go].unbind(1)
    remap[src] = dst
    new_refs[dst] = refs[src]
    new_refs[src] = 0
    j = torch.arange(st["tables"].shape[1], device=dev)
    t = st["tables"].long()
    new = torch.where(j < ((st["lens"].long() + bs - 1) // bs)[:, None], remap[t.clamp_min(0)], torch.full_like(t, -1))
    top = torch.where(new_refs > 0, b + 1, torch.zeros_like(b)).amax()
    _plain_copy(st, pairs)
    return dict(tables=new.to(torch.int32), refs=new_refs, remap=remap.to(torch.int32), pairs=pairs,
                status=torch.stack([go.sum(), U, top, moves]).to(torch.int32), k_cache=st["k_cache"],
                v_cache=st["v_cache"])


def _own_compact(st):
    from paged_kv_cache_251_gb300 import pa
    if "workspace" not in st:
        st["workspace"] = pa.pages_workspace_for(st["tables"], st["refs"])
    pa.pa_pages_compact(st["new_tables"], st["new_refs"], st["remap"], st["pairs"], st["status"], st["tables"],
                        st["refs"], st["lens"], block_size=st["case"]["block"], workspace=st["workspace"])
    pa.pa_copy_pages(st["pairs"], [st["k_cache"], st["v_cache"]])
    return dict(tables=st["new_tables"], refs=st["new_refs"], remap=st["remap"], pairs=st["pairs"],
                status=st["status"], k_cache=st["k_cache"], v_cache=st["v_cache"])


_PLAIN = dict(verify=_plain_verify, append=_plain_append, decode=_plain_decode, update=_plain_update,
              compact=_plain_compact)
_OWN = dict(verify=_own_verify, append=_own_append, decode=_own_decode, update=_own_update, compact=_own_compact)


# ---------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    if case["op"] == "verify":
        N, T, V, e = case["seqs"], case["draft"], case["vocab"], ELT[case["dtype"]]
        # the distributions behind the last accepted token, each drafted token's probabilities, the lists
        both = 2 if case["with_q"] else 1
        return dict(bytes=N * V * e * both + N * T * (e * both + 24) + 12 * N, flops=3 * N * V)
    bs, K, d = case["block"], case["kv_heads"], case["d"]
    if case["op"] == "append":
        lens = _lens(case["seqs"], case["min_len"], case["max_len"])
        T, e = sum(lens), ELT[case["dtype"]]
        blocks = sum(_up(n, bs) for n in lens)
        # rows read, codes written, a scale read and written for each block and head
        return dict(bytes=2 * T * K * d * (e + 1) + 8 * T + 16 * blocks * K, flops=4 * T * K * d)
    if case["op"] == "decode":
        N, H, e = case["seqs"], case["heads"], ELT[case["dtype"]]
        lens = _lens(N, case["min_len"], case["max_len"])
        toks = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        blocks = sum(_up(min(n, case["window"]) if case["window"] else n, bs) for n in lens)
        return dict(bytes=2 * toks * K * d + 8 * blocks * K + 4 * blocks + 2 * N * H * d * e + 4 * N,
                    flops=4 * toks * H * d)
    N = case["rows"]
    page = 2 * K * bs * d * ELT[case["dtype"]]
    if case["op"] == "update":
        B = case["beams"]
        lens = _lens(N // B, case["min_len"], case["max_len"])
        entries = B * sum(_up(n, bs) + _up(n + case["grow"], bs) for n in lens)
        # tables read and written, a count read and written for each block; a forked last block read and written
        forks = sum(n % bs != 0 for n in lens) * (B - 1)
        return dict(bytes=4 * entries + 8 * (entries // 2 // B) + 16 * N + 2 * page * forks, flops=0)
    lens = _lens(N, case["min_len"], case["max_len"])
    used, nb = sum(_up(n, bs) for n in lens), case["blocks"]
    moved = used * (nb - used) // nb
    return dict(bytes=8 * used + 12 * nb + 16 * (nb // 2) + 2 * page * moved, flops=0)


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return dict(verify=_exact_verify, append=_exact_append, decode=_exact_decode, update=_exact_update,
                compact=_exact_compact)[case["op"]](st)


def _exact_verify(st):
    P = st["target_probs"].double().cpu().numpy()
    Q = None if st["draft_probs"] is None else st["draft_probs"].double().cpu().numpy()
    tok, u = st["draft_tokens"].tolist(), st["uniforms"].double().cpu().numpy()
    N, T = len(tok), len(tok[0])
    parents = st["parents"].tolist() if st["parents"] is not None else [list(range(-1, T - 1))] * N
    lens, accepted, tokens = [], np.full((N, T), -1), np.full((N, T + 1), -1)
    for s, drafted in enumerate(st["draft_lens"].tolist()):
        path, node = [], -1
        w, total = P[s, 0], 1.0
        for i in range(drafted):
            if parents[s][i] != node:
                continue
            x = tok[s][i]
            if Q is None:
                took = u[s, i] * total < w[x]
            else:
                took = u[s, i] * total * Q[s, node + 1, x] < w[x]
            if took:
                path.append(i)
                node, w, total = i, P[s, i + 1], 1.0
            elif Q is None:
                total -= w[x]
                w = w.copy()
                w[x] = 0
            else:  # (w / total - q) up to a factor
                w = np.maximum(w - total * Q[s, node + 1], 0)
                total = w.sum()
        if not w.sum() > 0:
            w = P[s, node + 1]
        cum = np.cumsum(w)
        hit = np.nonzero(cum > u[s, T] * cum[-1])[0]
        x = int(hit[0]) if hit.size else int(np.nonzero(w > 0)[0][-1])
        lens.append(len(path))
        accepted[s, :len(path)] = path
        tokens[s, :len(path) + 1] = [tok[s][i] for i in path] + [x]
    return dict(accept_lens=torch.tensor(lens, dtype=torch.int32), accepted=torch.tensor(accepted, dtype=torch.int32),
                tokens=torch.tensor(tokens, dtype=torch.int32))


def _to_code(x, code):
    """The nearest code values of quotients that were rounded to 32 bits, ties to even, in 64 bits."""
    if code == "int8":
        return torch.round(x).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6, max=448.0))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(st):
    case, bs, top = st["case"], st["case"]["block"], QMAX[st["case"]["code"]]
    slots = st["slots"]
    out = {}
    for name in ("k", "v"):
        c, s = st[name + "_cache"].double(), st[name + "_scales"].double()
        x = st[name].double()
        order = torch.argsort(slots, stable=True)
        order = order[int((slots < 0).sum()):]
        blocks, counts = torch.unique_consecutive(slots[order] // bs, return_counts=True)
        # the rows of each touched block in a frame of its own, absent rows as NaN
        rows = torch.full((blocks.numel(), bs) + x.shape[1:], math.nan, dtype=torch.float64, device=x.device)
        which = torch.repeat_interleave(torch.arange(blocks.numel(), device=x.device), counts)
        rows[which, slots[order] % bs] = x[order]
        rows = rows.transpose(1, 2)  # block, head, row, d
        new = ~rows.isnan()
        peak = rows.nan_to_num(0).abs().amax((2, 3))
        want = (peak / top).float().double()  # the scale is held in 32 bits
        old = s[blocks]
        fresh = new[:, 0, 0, 0]
        scale = torch.where(fresh[:, None], want, torch.maximum(want, old))
        per = scale[:, :, None, None]
        again = (c[blocks] * old[:, :, None, None]).float().double()
        before = torch.where((scale > old)[:, :, None, None] & ~fresh[:, None, None, None],
                             _to_code((again / per).float().double(), case["code"]), c[blocks])
        coded = _to_code((rows.nan_to_num(0) / per).float().double(), case["code"])
        c[blocks] = torch.where(new, torch.where(per > 0, coded, torch.zeros_like(coded)), before)
        s[blocks] = scale
        out[name + "_cache"] = c if case["code"] == "e4m3" else c * s[:, :, None, None]
        out[name + "_scales"] = s
    return out


def _exact_decode(st):
    N, H, d = st["q"].shape
    K, bs, window = st["case"]["kv_heads"], st["case"]["block"], st["case"]["window"]
    out = torch.zeros((N, H, d), dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["lens"].tolist()):
        blocks = st["tables"][s, :_up(n, bs)].long()
        k, v = ((c[blocks].double() * f[blocks].double()[:, :, None, None]).transpose(1, 2).reshape(-1, K, d)[:n]
                for c, f in ((st["k_cache"], st["k_scales"]), (st["v_cache"], st["v_scales"])))
        first = max(0, n - window) if window else 0
        w = torch.einsum("kgd,nkd->kgn", st["q"][s].double().view(K, H // K, d), k[first:]) / math.sqrt(d)
        out[s] = torch.einsum("kgn,nkd->kgd", w.softmax(-1), v[first:]).reshape(H, d)
    return out


def _moved(st, pairs):
    out = {}
    for name in ("k_cache", "v_cache"):
        out[name] = st[name].double()
        if pairs:
            src, dst = torch.tensor(pairs, device="cuda").unbind(1)
            out[name][dst] = st[name][src].double()
    return out


def _exact_update(st):
    bs, tables, lens = st["case"]["block"], st["tables"].tolist(), st["lens"].tolist()
    parents, keep, grow = st["parents"].tolist(), st["keep"].tolist(), st["grow"].tolist()
    refs = st["refs"].tolist()
    N, M = len(tables), len(tables[0])
    for r in range(N):
        for b in tables[r][:_up(lens[r], bs)]:
            refs[b] -= 1
    held, ends = [], []
    for i in range(N):
        k = min(max(0, keep[i]), lens[parents[i]]) if parents[i] >= 0 else 0
        g = min(max(grow[i], k), M * bs)
        held.append(tables[parents[i]][:_up(k, bs)] if parents[i] >= 0 else [])
        ends.append((k, g))
        for b in held[i]:
            refs[b] += 1
    writers = {}
    for i, (k, g) in enumerate(ends):
        if g > k and k % bs:
            writers.setdefault(held[i][-1], []).append(i)
    copies = [i for b, who in writers.items() for i in who if not (len(who) == refs[b] and i == who[0])]
    copies = set(copies)
    need = [_up(g, bs) - _up(k, bs) + (i in copies) for i, (k, g) in enumerate(ends)]
    free = [b for b, n in enumerate(refs) if n == 0]
    spare = len(free)
    if sum(need) > spare:
        return None
    new, pairs = [], [(-1, -1)] * N
    for i in range(N):
        got, free = free[:need[i]], free[need[i]:]
        for b in got:
            refs[b] = 1
        row = list(held[i])
        if i in copies:
            refs[row[-1]] -= 1
            pairs[i] = (row[-1], got[0])
            row[-1] = got.pop(0)
        row += got
        new.append(row + [-1] * (M - len(row)))
    status = [1, sum(need), spare - sum(need), len(copies)]
    return dict(tables=torch.tensor(new, dtype=torch.int32), refs=torch.tensor(refs, dtype=torch.int32),
                pairs=torch.tensor(pairs), status=torch.tensor(status, dtype=torch.int32),
                **_moved(st, [p for p in pairs if p[0] >= 0]))


def _exact_compact(st):
    bs, refs, tables, lens = st["case"]["block"], st["refs"].tolist(), st["tables"].tolist(), st["lens"].tolist()
    nb, M = len(refs), len(tables[0])
    U = sum(n > 0 for n in refs)
    movers = [b for b in range(nb - 1, U - 1, -1) if refs[b] > 0]
    pairs = list(zip(movers, [b for b in range(U) if refs[b] == 0]))[:nb // 2]
    remap = list(range(nb))
    for a, b in pairs:
        remap[a], refs[b], refs[a] = b, refs[a], 0
    new = []
    for r, row in enumerate(tables):
        n = _up(lens[r], bs)
        new.append([remap[b] for b in row[:n]] + [-1] * (M - n))
    top = max([b + 1 for b in range(nb) if refs[b] > 0], default=0)
    return dict(tables=torch.tensor(new, dtype=torch.int32), refs=torch.tensor(refs, dtype=torch.int32),
                remap=torch.tensor(remap, dtype=torch.int32),
                pairs=torch.tensor(pairs + [(-1, -1)] * (nb // 2 - len(pairs))).reshape(-1, 2),
                status=torch.tensor([len(pairs), U, top, len(movers)], dtype=torch.int32), **_moved(st, pairs))
