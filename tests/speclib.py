"""64-bit oracles of the speculative and device-side operators' tests: plain numpy
or torch in float64, one sequence, block or row at a time, from the definitions."""
from __future__ import annotations

import numpy as np
import torch

QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


# ---------------------------------------------------------------------------
# Verification


def verify(target, draft, tokens, uniforms, lens=None, parents=None):
    """(accept_lens, accepted, tokens) of numpy float64 probabilities."""
    n, t = tokens.shape
    v = target.shape[2]
    out_n, out_a, out_t = np.zeros(n, int), np.full((n, t), -1), np.full((n, t + 1), -1)
    for s in range(n):
        drafted = t if lens is None else min(max(int(lens[s]), 0), t)
        node, path = -1, []
        w, total = np.maximum(np.nan_to_num(target[s, 0], nan=0.0), 0), 1.0
        gone = set()
        for i in range(drafted):
            parent = i - 1 if parents is None else int(parents[s, i])
            x = int(tokens[s, i])
            if parent >= i or not 0 <= x < v or max(parent, -1) != node:
                continue
            u = float(uniforms[s, i])
            if draft is None:
                took = x not in gone and u * total < w[x]
            else:
                took = u * total * draft[s, node + 1, x] < w[x]
            if took:
                path.append(i)
                node, total, gone = i, 1.0, set()
                w = np.maximum(np.nan_to_num(target[s, i + 1], nan=0.0), 0)
            elif draft is None:
                if x not in gone:
                    total -= w[x]
                    w = w.copy()
                    w[x] = 0
                    gone.add(x)
            else:
                w = w - total * draft[s, node + 1]
                w = np.where(w > 0, w, 0.0)  # (NaN: 0)
                total = w.sum()
        if not w.sum() > 0:
            w = np.maximum(np.nan_to_num(target[s, node + 1], nan=0.0), 0)
        cum = np.cumsum(w)
        x = -1
        if cum[-1] > 0:
            hit = np.nonzero(cum > float(uniforms[s, t]) * cum[-1])[0]
            x = int(hit[0]) if hit.size else int(np.nonzero(w > 0)[0][-1])
        out_n[s] = len(path)
        out_a[s, :len(path)] = path
        out_t[s, :len(path) + 1] = [int(tokens[s, i]) for i in path] + [x]
    return out_n, out_a, out_t


# ---------------------------------------------------------------------------
# Block-scaled caches


def nearest_code(x, dtype):
    """The value of the code nearest to each of x (float64, ties to even), NaN as 0."""
    x = torch.nan_to_num(x, nan=0.0, posinf=1e30, neginf=-1e30)
    if dtype == torch.int8:
        return torch.round(x).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6, max=448.0))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def f32(x):
    return x.float().double()


def append_block_quant(k, v, slots, kc, vc, ks, vs):
    """The cache after an append: float64 code values and scales, from CPU tensors."""
    bs = kc.shape[2]
    out = []
    for rows, cache, scales in ((k, kc, ks), (v, vc, vs)):
        q = QMAX[cache.dtype]
        c, s = cache.double(), scales.double()
        blocks = {}
        for i, slot in enumerate(slots.tolist()):
            if 0 <= slot < cache.shape[0] * bs:
                blocks.setdefault(slot // bs, {})[slot % bs] = i
        for b, where in blocks.items():
            at = sorted(where)
            x = rows[[where[r] for r in at]].double()  # [rows, heads, d]
            peak = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax((0, 2))
            mine = f32(peak / q)
            old = s[b].clone()
            fresh = 0 in where
            scale = mine if fresh else torch.maximum(mine, old)
            for h in range(cache.shape[1]):
                if not fresh and scale[h] > old[h]:
                    c[b, h] = nearest_code(f32(f32(c[b, h] * old[h]) / scale[h]), cache.dtype)
                for j, r in enumerate(at):
                    c[b, h, r] = nearest_code(f32(x[j, h] / scale[h]), cache.dtype) if scale[h] > 0 else 0.0
                s[b, h] = scale[h]
        out += [c, s]
    return out[0], out[2], out[1], out[3]


def decode_block_quant(q, kc, vc, ks, vs, tables, lens, scale=None, window=0):
    """Attention in float64 over code * scale, from CPU tensors; blocks outside the pool are left out."""
    n, h, d = q.shape
    nb, hkv, bs, _ = kc.shape
    scale = d ** -0.5 if scale is None else scale
    kc, vc = kc.double(), vc.double()
    out = torch.zeros((n, h, d), dtype=torch.float64)
    for s in range(n):
        length = min(max(int(lens[s]), 0), tables.shape[1] * bs)
        first = max(0, length - window) if window else 0
        toks = [t for t in range(first, length) if 0 <= int(tables[s, t // bs]) < nb]
        if not toks:
            continue
        b = torch.tensor([int(tables[s, t // bs]) for t in toks])
        r = torch.tensor([t % bs for t in toks])
        k = kc[b, :, r] * ks[b].double()[:, :, None]
        v = vc[b, :, r] * vs[b].double()[:, :, None]
        x = torch.einsum("kgd,nkd->kgn", q[s].double().view(hkv, h // hkv, d), k) * scale
        out[s] = torch.einsum("kgn,nkd->kgd", x.softmax(-1), v).reshape(h, d)
    return out


def block_pool(gen, blocks, hkv, bs, d, dtype, spread=0.5):
    """Random codes and scales as an append leaves them (CPU)."""
    top = QMAX[dtype]
    x = (torch.randn((blocks, hkv, bs, d), generator=gen) * (top / 3.5)).clamp(-top, top)
    codes = x.round().to(torch.int8) if dtype == torch.int8 else x.to(dtype)
    scales = torch.exp(spread * torch.randn((blocks, hkv), generator=gen)) * (3.5 / top)
    return codes, scales


# ---------------------------------------------------------------------------
# Page tables


def pages_update(tables, refs, lens, parents, keep, grow, bs):
    """(new tables, refs, pairs, status) from lists; tables and refs None when the blocks do not suffice."""
    up = lambda x: -(-x // bs)  # noqa: E731
    nb, m = len(refs), len(tables[0]) if tables else 0
    refs = list(refs)
    cap = m * bs
    lens = [min(max(x, 0), cap) for x in lens]
    inside = lambda b: 0 <= b < nb  # noqa: E731
    for r, row in enumerate(tables):
        for b in row[:up(lens[r])]:
            if inside(b):
                refs[b] -= 1
    rows = []
    for i in range(len(keep)):
        p = parents[i] if parents is not None else i
        p = p if 0 <= p < len(tables) else -1
        k = min(max(keep[i], 0), lens[p]) if p >= 0 else 0
        g = min(max(grow[i], k), cap)
        held = list(tables[p][:up(k)]) if p >= 0 else []
        for b in held:
            if inside(b):
                refs[b] += 1
        rows.append((k, g, held))
    writers = {}
    for i, (k, g, held) in enumerate(rows):
        if g > k and k % bs and inside(held[-1]):
            writers.setdefault(held[-1], []).append(i)
    copied = set()
    for b, who in writers.items():
        copied.update(who if len(who) != refs[b] else who[1:])
    need = [up(g) - up(k) + (i in copied) for i, (k, g, _) in enumerate(rows)]
    free = [b for b in range(nb) if refs[b] == 0]
    pairs = [[-1, -1] for _ in rows]
    if sum(need) > len(free):
        return None, None, pairs, [0, sum(need), len(free), 0]
    left = iter(free)
    new = []
    for i, (k, g, held) in enumerate(rows):
        if i in copied:
            dst = next(left)
            refs[dst] = 1
            refs[held[-1]] -= 1
            pairs[i] = [held[-1], dst]
            held[-1] = dst
        while len(held) < up(g):
            b = next(left)
            refs[b] = 1
            held.append(b)
        new.append(held + [-1] * (m - len(held)))
    return new, refs, pairs, [1, sum(need), len(free) - sum(need), len(copied)]


def pages_compact(tables, refs, lens, bs, max_moves):
    """(new tables, refs, remap, pairs, status) from lists."""
    nb, m = len(refs), len(tables[0]) if tables else 0
    refs = list(refs)
    used = sum(x > 0 for x in refs)
    movers = [b for b in range(nb - 1, used - 1, -1) if refs[b] > 0]
    holes = [b for b in range(used) if refs[b] <= 0]
    pairs = [list(x) for x in zip(movers, holes)][:max_moves]
    remap = list(range(nb))
    for a, b in pairs:
        remap[a] = b
        refs[b], refs[a] = refs[a], 0
    new = []
    for row, n in zip(tables, lens):
        n = -(-min(max(n, 0), m * bs) // bs)
        new.append([remap[b] if 0 <= b < nb else b for b in row[:n]] + [-1] * (m - n))
    top = max([b + 1 for b in range(nb) if refs[b] > 0], default=0)
    status = [len(pairs), used, top, len(movers)]
    return new, refs, remap, pairs + [[-1, -1]] * (max_moves - len(pairs)), status
