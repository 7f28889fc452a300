"""The block-scaled 8-bit cache: append bit for bit against the definition, decode
against attention in 64 bits over code * scale."""
import math

import pytest
import torch

import speclib
from paged_kv_cache_251_gb300 import pa

pytestmark = pytest.mark.gpu

I8, E4M3 = torch.int8, torch.float8_e4m3fn


def same_cache(got, want):
    kc, vc, ks, vs = got
    for g, w in zip((ks, vs, kc, vc), (want[2], want[3], want[0], want[1])):
        assert torch.equal(g.cpu().double(), w)


def append(k, v, slots, kc, vc, ks, vs, **more):
    dev = [x.cuda().clone() for x in (kc, vc, ks, vs)]
    pa.pa_append_kv_block_quant(k.cuda(), v.cuda(), slots.cuda(), *dev, **more)
    torch.cuda.synchronize()
    return dev


def rows(gen, n, hkv, d, dtype, spread=1.0):
    size = torch.exp(spread * torch.randn((n, hkv, 1), generator=gen))
    return (torch.randn((n, hkv, d), generator=gen) * size).to(dtype)


def pool(gen, nb, hkv, bs, d, code):
    kc, ks = speclib.block_pool(gen, nb, hkv, bs, d, code)
    vc, vs = speclib.block_pool(gen, nb, hkv, bs, d, code)
    return kc, vc, ks, vs


def check_append(gen, n, hkv, d, bs, nb, code, dtype, slots, spread=1.0):
    cache = pool(gen, nb, hkv, bs, d, code)
    k, v = rows(gen, n, hkv, d, dtype, spread), rows(gen, n, hkv, d, dtype, spread)
    got = append(k, v, slots, *cache)
    want = speclib.append_block_quant(k, v, slots, *cache)
    same_cache(got, want)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128), (8, 128)])
def test_append_scattered(code, dtype, bs, hkv, d):
    """Slots in no order, several or all rows of some blocks, padding, with and without row 0."""
    gen = torch.Generator().manual_seed(bs + hkv)
    nb = 9
    slots = torch.randperm(nb * bs, generator=gen)[:nb * bs // 3]
    slots[::7] = -1
    check_append(gen, slots.numel(), hkv, d, bs, nb, code, dtype, slots)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("n", [1, 2, 511, 512, 513, 1300])
def test_append_by_number_of_tokens(code, n):
    gen = torch.Generator().manual_seed(n)
    nb = n // 16 + 40
    start = torch.randint(0, 16, (1,), generator=gen).item()
    contiguous = torch.randperm(nb, generator=gen)[torch.arange(start, start + n) // 16] * 16 + \
        torch.arange(start, start + n) % 16
    for slots in (contiguous, torch.randperm(nb * 16, generator=gen)[:n], contiguous.flip(0).contiguous()):
        check_append(gen, n, 2, 128, 16, nb, code, torch.bfloat16, slots)


def test_append_grows_a_block_token_by_token():
    """Every row of a block by a call of its own: the scale only grows, row 0 starts anew."""
    gen = torch.Generator().manual_seed(3)
    cache = list(pool(gen, 3, 2, 16, 64, I8))
    for turn in range(2):
        for r in range(16):
            k, v = rows(gen, 1, 2, 64, torch.float32, 2.0), rows(gen, 1, 2, 64, torch.float32, 2.0)
            slots = torch.tensor([16 + r])
            before = cache[2][1].clone()
            got = append(k, v, slots, *cache)
            same_cache(got, speclib.append_block_quant(k, v, slots, *cache))
            cache = [x.cpu() for x in got]
            assert r == 0 or (cache[2][1] >= before).all()


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("n", [5, 600])
def test_append_special_values(code, n):
    """Zeros, infinities, NaN, the smallest and largest numbers; a block of zeros has scale 0."""
    gen = torch.Generator().manual_seed(4)
    nb = n // 16 + 3
    cache = pool(gen, nb, 2, 16, 64, code)
    cache[2][1] = 0
    k, v = rows(gen, n, 2, 64, torch.float32), rows(gen, n, 2, 64, torch.float32)
    slots = torch.arange(n) + 3
    k[0], v[1] = 0, 0
    k[1, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e-44])
    v[2, 1] = float("nan")
    v[3, 0, 5] = 3.4e38
    k[4] = 1e-42
    got = append(k, v, slots, *cache)
    same_cache(got, speclib.append_block_quant(k, v, slots, *cache))
    zero = append(torch.zeros(16, 2, 64), torch.zeros(16, 2, 64), torch.arange(16), *cache)
    assert (zero[2][0] == 0).all() and (zero[0][0].float() == 0).all()


def test_append_bad_slots_and_duplicates():
    gen = torch.Generator().manual_seed(5)
    cache = pool(gen, 4, 2, 16, 64, I8)
    k = rows(gen, 6, 2, 64, torch.float32)
    slots = torch.tensor([5, 64, -1, 1 << 40, -(1 << 40), 20])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = append(k, k, slots, *cache, err_word=err)
    assert err.item() == pa.DEVERR_BAD_SLOT
    same_cache(got, speclib.append_block_quant(k, k, slots, *cache))
    for n in (3, 700):  # one slot named twice: one of the rows, whole, and a scale that fits it
        slots = torch.arange(n) % 64
        slots[n - 1] = slots[n - 2]
        k = rows(gen, n, 2, 64, torch.float32)
        got = append(k, k, slots, *cache) if n == 3 else None
        if got is not None:
            one = [append_one(k[[0, j]], torch.tensor([0, 1]), cache) for j in (1, 2)]
            assert any(all(torch.equal(a, b) for a, b in zip(got, w)) for w in one)


def append_one(k, slots, cache):
    return append(k, k, slots, *cache)


def test_append_nothing_and_untouched_blocks():
    gen = torch.Generator().manual_seed(6)
    cache = pool(gen, 4, 2, 16, 128, E4M3)
    none = torch.empty(0, 2, 128)
    got = append(none, none, torch.empty(0, dtype=torch.int64), *cache)
    assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, cache))
    pad = rows(gen, 700, 2, 128, torch.float32)
    got = append(pad, pad, torch.full((700,), -1), *cache)
    assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, cache))


def test_append_workspace_of_any_contents():
    gen = torch.Generator().manual_seed(7)
    n, nb = 900, 80
    cache = pool(gen, nb, 1, 16, 64, I8)
    k = rows(gen, n, 1, 64, torch.float16)
    slots = torch.randperm(nb * 16, generator=gen)[:n]
    slots[100:200] = -1
    want = speclib.append_block_quant(k, k, slots, *cache)
    for fill in (0, -1, 899, 2**31 - 1, -2**31):
        ws = torch.full((nb * 16 + nb + 1,), fill, dtype=torch.int32, device="cuda")
        same_cache(append(k, k, slots, *cache, workspace=ws), want)
    ws = torch.arange(nb * 17 + 1, dtype=torch.int32, device="cuda") % n
    same_cache(append(k, k, slots, *cache, workspace=ws), want)


@pytest.mark.parametrize("n,hkv", [(40, 300), (520, 1900)])
def test_append_more_heads_than_warps(n, hkv):
    """Units beyond the warps that share them: each head's codes are those of a call with it alone."""
    gen = torch.Generator().manual_seed(41)
    nb = 40
    cache = pool(gen, nb, 1, 16, 64, I8)
    cache = [x.expand(-1, hkv, *x.shape[2:]).contiguous() for x in cache]
    k, v = (rows(gen, n, 1, 64, torch.bfloat16).expand(n, hkv, 64).clone() for _ in range(2))
    some = [0, 1, hkv // 2, hkv - 2, hkv - 1]
    for h in some:
        k[:, h], v[:, h] = rows(gen, n, 1, 64, torch.bfloat16)[:, 0], rows(gen, n, 1, 64, torch.bfloat16)[:, 0]
    slots = torch.randperm(nb * 16, generator=gen)[:n]
    got = append(k, v, slots, *cache)
    for part in (some, [2]):
        sub = [x[:, part].contiguous() for x in cache]
        same_cache([x[:, part] for x in got],
                   speclib.append_block_quant(k[:, part].contiguous(), v[:, part].contiguous(), slots, *sub))
    rest = [h for h in range(hkv) if h not in some]  # (all alike)
    for x in got:
        assert (x[:, rest] == x[:, [2]]).all()


def test_append_streams_graphs_and_one_workspace_after_another():
    gen = torch.Generator().manual_seed(42)
    nb, n = 150, 2000
    cache = [x.cuda() for x in pool(gen, nb, 3, 32, 128, E4M3)]
    slots = torch.randperm(nb * 32, generator=gen)[:n]
    slots[::9] = -1
    k, v = rows(gen, n, 3, 128, torch.float16), rows(gen, n, 3, 128, torch.float16)
    want = speclib.append_block_quant(k, v, slots, *[x.cpu() for x in cache])
    dev = [k.cuda(), v.cuda(), slots.cuda()]
    ws = pa.append_block_quant_workspace_for(dev[2], cache[0])
    copies = [[x.clone() for x in cache] for _ in range(4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_append_kv_block_quant(*dev, *copies[0], workspace=ws)
    pa.pa_append_kv_block_quant(*dev, *copies[1], stream=side)
    other = slots.flip(0).contiguous().cuda()  # the workspace holds another call's map
    pa.pa_append_kv_block_quant(dev[0].flip(0).contiguous(), dev[1].flip(0).contiguous(), other, *copies[2], workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_append_kv_block_quant(*dev, *copies[3], workspace=ws)
    ws.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for got in copies:
        same_cache(got, want)
    graph.replay()  # the same rows again: scales stay or, where row 0 is among them, are set anew alike
    torch.cuda.synchronize()
    again = speclib.append_block_quant(k, v, slots, *[x.cpu() for x in copies[0]])
    same_cache(copies[3], again)


# ---------------------------------------------------------------------------
# Decode.  Beside half a step of the output's type, an output row's error is bounded
# by the arithmetic: scores are fp32 sums of d products (relative to sum |q k|: about
# d / 2 * 2^-24 at worst, exact products), the exponential is good to 2^-22, weights are
# kept to 22 bits, and sums over L tokens lose 2^-24 a step at most.  In units of the
# largest |v| of a row: TOL below covers them with scores up to 40 (an error of the
# score, 64 * 2^-24 * 40, is a relative one of the weight).

TOL = 64 * 40 * 2.0 ** -24 + 2.0 ** -21


def paged(gen, lens, hkv, bs, d, code, extra=3, width=None):
    need = [(n + bs - 1) // bs for n in lens]
    nb = sum(need) + extra
    order = torch.randperm(nb, generator=gen)
    tables = torch.full((len(lens), width or max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n].int()
        at += n
    return pool(gen, nb, hkv, bs, d, code) + (tables, torch.tensor(lens, dtype=torch.int32))


def check_decode(q, cache, out_dtype=None, window=0, scale=None, err=None, **more):
    out_dtype = out_dtype or q.dtype
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    pa.pa_decode_block_quant(out, q.cuda(), *[x.cuda() for x in cache], window=window, scale=scale, err_word=err,
                             **more)
    torch.cuda.synchronize()
    want = speclib.decode_block_quant(q, *cache, scale=scale, window=window)
    got = out.cpu().double()
    top = (cache[1].double().abs().amax((2, 3)) * cache[3].double()).nan_to_num(0).amax().item()
    half = torch.finfo(out_dtype).eps / 2
    tiny = torch.finfo(out_dtype).smallest_normal * torch.finfo(out_dtype).eps
    assert got.isfinite().all()
    far = (got - want).abs() - (TOL * top + half * want.abs() * (1 + half) + tiny)
    assert far.max() <= 0, (far.max().item(), (got - want).abs().max().item())
    return out


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_decode_shapes(code, dtype, bs, d, group):
    gen = torch.Generator().manual_seed(group)
    lens = [1, 0, 7, 8, 9, 16, 17, 31, 33, 130, 500]
    cache = paged(gen, lens, 2, bs, d, code)
    q = torch.randn((len(lens), 2 * group, d), generator=gen).to(dtype)
    check_decode(q, cache, out_dtype=torch.float32)
    check_decode(q, cache)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("bs,d,group", [(8, 128, 4), (16, 64, 1), (16, 128, 8), (32, 128, 2), (32, 64, 8)])
def test_decode_long_and_ragged(code, bs, d, group):
    """Contexts cut between warps, CTAs, many CTAs."""
    gen = torch.Generator().manual_seed(20)
    for lens in ([20000], [3, 9000, 0, 1, 700, 4097], [300] * 70):
        cache = paged(gen, lens, 1 if len(lens) < 50 else 2, bs, d, code)
        q = torch.randn((len(lens), (1 if len(lens) < 50 else 2) * group, d), generator=gen).to(torch.float16)
        check_decode(q, cache, out_dtype=torch.float32)


def test_decode_many_sequences():
    gen = torch.Generator().manual_seed(21)
    lens = torch.randint(0, 60, (700,), generator=gen).tolist()
    cache = paged(gen, lens, 1, 16, 64, I8)
    check_decode(torch.randn((700, 4, 64), generator=gen).to(torch.bfloat16), cache, out_dtype=torch.float32)


@pytest.mark.parametrize("window", [1, 5, 16, 33, 250, 100000])
@pytest.mark.parametrize("bs,d", [(8, 64), (16, 128), (32, 64)])
def test_decode_window(window, bs, d):
    gen = torch.Generator().manual_seed(22)
    cache = list(paged(gen, [1, 6, 40, 251, 1000], 2, bs, d, E4M3))
    for s, n in enumerate((1, 6, 40, 251, 1000)):  # entries before the window are not read
        cache[4][s, :max(0, n - window) // bs] = 1 << 30
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_decode(torch.randn((5, 8, d), generator=gen), cache, window=window, err=err)
    assert err.item() == 0


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("size", [1e-30, 1e-4, 30.0, 1e4])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_query_sizes(code, size, dtype):
    """Queries of any size: the scale puts the scores back."""
    gen = torch.Generator().manual_seed(23)
    cache = paged(gen, [100, 333], 2, 16, 128, code)
    q = (torch.randn((2, 8, 128), generator=gen) * size).to(dtype)
    check_decode(q, cache, out_dtype=torch.float32, scale=128 ** -0.5 / size)


def test_decode_queries_of_wide_range():
    """Elements of 1e-3 to 1e3 in a row, the keys of the large ones cleared."""
    gen = torch.Generator().manual_seed(24)
    cache = paged(gen, [400], 1, 16, 128, I8)
    q = torch.randn((1, 4, 128), generator=gen)
    q[:, :, 5] = 1000.0
    q[:, :, 6:20] *= 1e-3
    cache[0][:, :, :, 5] = 0
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        check_decode(q.to(dtype), cache, out_dtype=torch.float32)


@pytest.mark.parametrize("group", [1, 4, 8])
def test_decode_peaked_and_ramped_scores(group):
    """The running maximum moves in every tile, up and down; far weights keep their mass."""
    gen = torch.Generator().manual_seed(25)
    for step in (0.04, -0.04, 2.0):
        n = 900
        kc, vc, ks, vs, tables, lens = paged(gen, [n], 1, 16, 64, I8)
        kc.zero_()
        # the score of token t is step * t: one key element ramps in its block's scale and code
        for t in range(n):
            b = int(tables[0, t // 16])
            kc[b, 0, t % 16, 0] = 100
        q = torch.zeros((1, group, 64))
        q[:, :, 0] = 1.0
        base = torch.arange((n + 15) // 16) * 16.0
        ks[tables[0].long(), 0] = base * step / 100
        check_decode(q, (kc, vc, ks, vs, tables, lens), out_dtype=torch.float32, scale=1.0)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[40], [5000, 40]])
def test_decode_scores_far_below_zero(code, dtype, lens):
    """All scores at or below -1e30: the largest of them, 1e30 above the next, takes all the weight."""
    kc, vc, ks, vs, tables, _ = cache = paged(torch.Generator().manual_seed(40), lens, 1, 16, 64, code)
    kc.zero_()
    kc[:, :, :, 0] = 2
    ks.fill_(1.0)
    q = torch.zeros((len(lens), 4, 64))
    q[:, :, 0] = -1e30
    best = [n * 2 // 3 for n in lens]
    for s, at in enumerate(best):
        kc[int(tables[s, at // 16]), 0, at % 16, 0] = 1
    out = check_decode_raw(q.to(dtype), cache, scale=1.0)
    for s, at in enumerate(best):
        b = int(tables[s, at // 16])
        want = vc[b, 0, at % 16].double() * vs[b, 0].double()
        # (the weight is 1 exactly; it and V's scale are rounded to 22 bits, the result to dtype)
        bound = want.abs() * (2.0 ** -20 + torch.finfo(dtype).eps / 2)
        assert ((out[s].cpu().double() - want).abs() <= bound).all()


def test_decode_small_weights_add_up():
    """8192 tokens 20 powers of two below one: together they weigh 2^-7 of it."""
    kc, vc, ks, vs, tables, lens = paged(torch.Generator().manual_seed(26), [8193], 1, 16, 64, I8)
    kc.zero_(), vc.zero_()
    ks.fill_(1.0), vs.fill_(1.0)
    first = int(tables[0, 0])
    kc[first, 0, 0, 0] = 20
    vc[:, :, :, 1] = 64
    vc[first, 0, 0, 1] = 0
    q = torch.zeros((1, 1, 64))
    q[:, :, 0] = math.log(2.0)
    out = torch.empty((1, 1, 64), device="cuda")
    pa.pa_decode_block_quant(out, q.cuda(), *[x.cuda() for x in (kc, vc, ks, vs, tables, lens)], scale=1.0)
    want = 64 * 8192 * 2.0 ** -20 / (1 + 8192 * 2.0 ** -20)
    assert abs(out[0, 0, 1].item() - want) <= want * 2.0 ** -16


def test_decode_blocks_outside_the_pool():
    gen = torch.Generator().manual_seed(27)
    cache = list(paged(gen, [100, 64, 33], 2, 16, 64, I8))
    cache[4][0, 2] = 1 << 29
    cache[4][1] = -5
    cache[2][0], cache[3][0] = float("nan"), float("nan")  # block 0 stands in for the bad ones
    used = cache[4][(cache[4] > 0) & (cache[4] < 1 << 29)]
    cache[4] = torch.where(cache[4] == 0, int(used[0]), cache[4])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = check_decode(torch.randn((3, 4, 64), generator=gen), cache, err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK and (out[1] == 0).all()


@pytest.mark.parametrize("bs", [8, 16, 32])
def test_decode_rows_behind_the_context(bs):
    """Codes behind the context, E4M3 NaN among them, and unused blocks' scales have no influence."""
    gen = torch.Generator().manual_seed(28)
    lens = [1, 13, 70]
    cache = list(paged(gen, lens, 2, bs, 128, E4M3))
    q = torch.randn((3, 8, 128), generator=gen).to(torch.float16)
    want = check_decode(q, cache)
    spoiled = [x.clone() for x in cache]
    used = torch.zeros(cache[0].shape[0], dtype=torch.bool)
    for s, n in enumerate(lens):
        b = int(cache[4][s, (n - 1) // bs])
        used[cache[4][s, :(n + bs - 1) // bs].long()] = True
        for c in spoiled[:2]:
            c.view(torch.uint8)[b, :, n - (n - 1) // bs * bs:] = 0x7f
    for c in spoiled[2:4]:
        c[~used] = float("nan")
    assert torch.equal(check_decode_raw(q, spoiled), want)


def check_decode_raw(q, cache, **more):
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    pa.pa_decode_block_quant(out, q.cuda(), *[x.cuda() for x in cache], **more)
    torch.cuda.synchronize()
    return out


def test_decode_context_longer_than_the_table():
    gen = torch.Generator().manual_seed(29)
    cache = list(paged(gen, [64, 20], 1, 16, 64, I8))
    q = torch.randn((2, 2, 64), generator=gen)
    want = check_decode_raw(q, cache)
    cache[5][0] = 70
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(check_decode_raw(q, cache, err_word=err), want) and err.item() == pa.DEVERR_BAD_LEN
    cache[5][1] = -3
    assert (check_decode_raw(q, cache)[1] == 0).all()


def test_decode_nan_stays_in_its_row():
    gen = torch.Generator().manual_seed(30)
    cache = paged(gen, [50, 3000], 2, 16, 128, I8)
    q = torch.randn((2, 8, 128), generator=gen)
    want = check_decode_raw(q, cache)
    q[1, 3, 7] = float("nan")
    got = check_decode_raw(q, cache)
    assert got[1, 3].isnan().all()
    got[1, 3] = want[1, 3]
    assert torch.equal(got, want)


def test_decode_same_bits_streams_graphs_workspaces():
    gen = torch.Generator().manual_seed(31)
    cache = [x.cuda() for x in paged(gen, [3000, 17, 900, 0], 2, 16, 128, E4M3)]
    q = torch.randn((4, 8, 128), generator=gen).to(torch.bfloat16).cuda()
    want = torch.empty_like(q)
    pa.pa_decode_block_quant(want, q, *cache)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.empty_like(q) for _ in range(4)]
    for i in range(20):
        pa.pa_decode_block_quant(outs[0], q, *cache)
        pa.pa_decode_block_quant(outs[1], q, *cache, stream=side)
    ws = pa.block_quant_workspace_for(q, cache[0], cache[4].shape[1])
    pa.pa_decode_block_quant(outs[2], q, *cache, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_block_quant(outs[3], q, *cache, workspace=ws)
    ws.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


def test_decode_large_offsets():
    """Blocks beyond 2^31 bytes from the pool's start."""
    gen = torch.Generator().manual_seed(32)
    nb, hkv, bs, d = 80000, 8, 32, 128  # 2.6 GB of codes each
    small = pool(gen, 6, hkv, bs, d, I8)
    at = torch.tensor([79999, 65537, 70001, 3, 78000, 66000])
    kc = torch.zeros((nb, hkv, bs, d), dtype=I8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = (torch.zeros((nb, hkv), device="cuda") for _ in range(2))
    for big, part in zip((kc, vc, ks, vs), small):
        big[at.cuda()] = part.cuda()
    q = torch.randn((2, 32, d), generator=gen)
    tables, lens = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32), torch.tensor([90, 96], dtype=torch.int32)
    want = speclib.decode_block_quant(q, *small, tables, lens)
    out = torch.empty(q.shape, device="cuda")
    pa.pa_decode_block_quant(out, q.cuda(), kc, vc, ks, vs, at[tables.long()].int().cuda(), lens.cuda())
    assert (out.cpu().double() - want).abs().max() <= TOL * 40
    rows_ = torch.randn((2, hkv, d), generator=gen)
    slots = torch.tensor([79999 * bs + 31, 65537 * bs])
    pa.pa_append_kv_block_quant(rows_.cuda(), rows_.cuda(), slots.cuda(), kc, vc, ks, vs)
    torch.cuda.synchronize()
    where = torch.tensor([31, 32])
    want = speclib.append_block_quant(rows_, rows_, where, *small)
    for got, w in zip((kc, vc, ks, vs), (want[0], want[1], want[2], want[3])):
        assert torch.equal(got[at.cuda()].cpu().double(), w)
