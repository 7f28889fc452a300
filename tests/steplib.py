"""64-bit oracles and derived bounds for the serving-step operators' tests:
plain torch in float64, one sequence at a time, from the definitions."""
from __future__ import annotations

import math

import torch

from paged_kv_cache_251_gb300 import workloads as wl

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def paged(seed, lens, hkv, d, bs, dtype, device="cuda", extra_blocks=3, max_blocks=None):
    """A shuffled paged cache holding the given context lengths: k_cache,
    v_cache, tables (int32, unused entries -1), lens (int32)."""
    need = [(n + bs - 1) // bs for n in lens]
    nb = sum(need) + extra_blocks
    width = max_blocks or max(max(need), 1)
    order = wl.permutation(seed, 2, nb).to(torch.int32)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    k = wl.normal_tensor(seed, 4, (nb, hkv, bs, d), dtype=dtype)
    v = wl.normal_tensor(seed, 5, (nb, hkv, bs, d), dtype=dtype)
    return (k.to(device), v.to(device), tables.to(device),
            torch.tensor(lens, dtype=torch.int32, device=device))


def rows_of(cache, table, n):
    """The first n cached rows of a sequence [n, H_kv, d], float64."""
    bs = cache.shape[2]
    if n == 0:
        return torch.zeros((0, cache.shape[1], cache.shape[3]), dtype=torch.float64, device=cache.device)
    b = table[:(n + bs - 1) // bs].long()
    return cache[b].transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[:n].double()


def random_parents(seed, n, t):
    u = wl.uniform01(seed, 11, n * t).view(n, t)
    return (u * (torch.arange(t) + 1)).floor().long() - 1


def attend(q, k, v, allowed, scale):
    """Attention of q [R, K, G, d] over k, v [n, K, d] with allowed bool [R, n]
    (masked rows of k and v never enter): (out, sum w |v|, score error bound, w).

    The score error bound is that of an fp32 dot product of d exact products
    (any order of summation): (d + 2) u sum |q_j k_j| scale."""
    R, K, G, d = q.shape
    out = torch.zeros_like(q)
    mag = torch.zeros_like(q)
    dx = torch.zeros((R, K, G), dtype=torch.float64, device=q.device)
    w_all = torch.zeros((R, K, G, k.shape[0]), dtype=torch.float64, device=q.device)
    for r in range(R):
        at = allowed[r].nonzero()[:, 0]
        if at.numel() == 0:
            continue
        kr, vr = k[at], v[at]
        x = torch.einsum("kgd,nkd->kgn", q[r], kr) * scale
        w = torch.softmax(x, -1)
        out[r] = torch.einsum("kgn,nkd->kgd", w, vr)
        mag[r] = torch.einsum("kgn,nkd->kgd", w, vr.abs())
        dx[r] = (torch.einsum("kgd,nkd->kgn", q[r].abs(), kr.abs()) * abs(scale)).amax(-1) * (d + 2) * U32
        w_all[r][:, :, at] = w
    return out, mag, dx, w_all


def tree_allowed(n, drafted, t, mask_row, device):
    """allowed [t, n] of one sequence: committed tokens, and drafted token j when
    mask_row says so for query i (mask_row None: j <= i)."""
    a = torch.zeros((t, n), dtype=torch.bool)
    for i in range(drafted):
        a[i, :n - drafted] = True
        for j in range(drafted):
            if mask_row is None:
                on = j <= i
            else:
                on = (int(mask_row[i, j // 64]) >> (j % 64)) & 1
            a[i, n - drafted + j] = bool(on)
    return a.to(device)


def tree_oracle(q, k_cache, v_cache, tables, lens, drafts, mask, scale):
    """(out, bound ingredients) of pa_decode_tree in float64."""
    N, T, H, d = q.shape
    K = k_cache.shape[1]
    out = torch.zeros((N, T, H, d), dtype=torch.float64, device=q.device)
    mag, dx = torch.zeros_like(out), torch.zeros((N, T, H), dtype=torch.float64, device=q.device)
    for s in range(N):
        n, td = int(lens[s]), int(drafts[s])
        k, v = rows_of(k_cache, tables[s], n), rows_of(v_cache, tables[s], n)
        allowed = tree_allowed(n, td, T, None if mask is None else mask[s].cpu(), q.device)
        o, m, e, _ = attend(q[s].double().view(T, K, H // K, d), k, v, allowed, scale)
        out[s], mag[s], dx[s] = o.reshape(T, H, d), m.reshape(T, H, d), e.reshape(T, H)
    return out, mag, dx


def weight_half_step(kv_dtype, out_dtype) -> float:
    """Relative rounding of a softmax weight before the P V product.  fp32
    caches: none.  16-bit caches: one rounding to the cache's type where the
    output is rounded to 16 bits anyway, two parts (hi + lo) for fp32 output."""
    if kv_dtype == torch.float32:
        return 0.0
    h = half_step(kv_dtype)
    return h * h if out_dtype == torch.float32 else h


def attention_bound(ref, mag, dx, kv_dtype, out_dtype, tokens):
    """Elementwise bound of an attention output: the output's rounding, the
    weights' rounding, the scores' error (a weight e^x moves by 2 dx relative,
    numerator and denominator together), the exponential (2^-21 covers
    ex2.approx's 2 ulp and the scaled argument's rounding for |x| < 2^7 in
    base-2 units: 2^7 u ln 2), and fp32 sums of `tokens` terms in tiles and
    running rescales (relative to sum w |v|)."""
    arg = 2.0 ** -21 + 2.0 ** 7 * U32
    sums = (math.sqrt(max(tokens, 1)) + 16) * 2 * U32
    rel = weight_half_step(kv_dtype, out_dtype) + 2 * dx[..., None] + arg + sums
    tiny = 2.0 ** -25 if out_dtype == torch.float16 else 0.0
    return half_step(out_dtype) * (ref.abs() + rel * mag) + rel * mag + tiny


def check_within(got, ref, bound, what=""):
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    over = (g - ref).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {float((g - ref).abs().flatten()[over.argmax()]):.3e} off, bound " \
                       f"{float(bound.flatten()[over.argmax()]):.3e}"
