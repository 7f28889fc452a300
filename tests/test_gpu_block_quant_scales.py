"""pa_decode_block_quant over V scales of very different sizes: what a block contributes must not hang on
its neighbours' scales, in whatever order they come.

A row's error is bounded as in test_gpu_block_quant.py, but in units of what its own tokens weigh:
M = sum p_t max |v_t| (and three times as large: TOL is for scores up to 40, here they reach 110), with
what the kernel loses below 2^-80 of the largest |v| beside it."""
import itertools

import pytest
import torch

import speclib
from paged_kv_cache_251_gb300 import pa
from test_gpu_block_quant import E4M3, I8, TOL, check_decode, paged

pytestmark = pytest.mark.gpu

FORMS = [(8, 64, 4), (8, 64, 8), (8, 128, 2), (8, 128, 8), (16, 64, 1), (16, 64, 8), (16, 128, 4), (16, 128, 8),
         (32, 64, 4), (32, 64, 8)]


def decode(q, cache, scale=None):
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pa.pa_decode_block_quant(out, q.cuda(), *[x.cuda() for x in cache], scale=scale)
    torch.cuda.synchronize()
    return out.cpu().double()


def check_rows(q, cache):
    got, want = decode(q, cache), speclib.decode_block_quant(q, *cache)
    ones = torch.ones_like(cache[1].float()).to(cache[1].dtype)
    weighed = speclib.decode_block_quant(q, cache[0], ones, cache[2], cache[3].abs() * speclib.QMAX[cache[1].dtype],
                                         *cache[4:])
    largest = cache[3].double().abs().max() * speclib.QMAX[cache[1].dtype]
    assert got.isfinite().all()
    far = (got - want).abs() - (3 * TOL * weighed + 2.0 ** -80 * largest + 2.0 ** -24 * want.abs() + 2.0 ** -140)
    assert far.max() <= 0, ((got - want).abs() / weighed).max().item()


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("bs,d,group", FORMS)
@pytest.mark.parametrize("sizes", [(0.03, 1e-36, 0.02, 1e-38), (1e-36, 1e-20, 1.0, 1e20)])
def test_scales_in_every_order(code, bs, d, group, sizes):
    """24 sequences, one for each order of four sizes, each over two to five blocks."""
    gen = torch.Generator().manual_seed(bs + d + group)
    orders = list(itertools.permutations(sizes))
    lens = torch.randint(12 * bs, 17 * bs, (24,), generator=gen).tolist()
    cache = list(paged(gen, lens, 2, bs, d, code))
    for s, order in enumerate(orders):
        cuts = torch.randint(2, 6, (4,), generator=gen).tolist()
        per_block = (sum(([x] * n for x, n in zip(order, cuts)), []) + [order[3]] * 20)[:-(-lens[s] // bs)]
        b = cache[4][s, :len(per_block)].long()
        cache[3][b] = torch.tensor(per_block)[:, None] * (0.5 + torch.rand((len(per_block), 2), generator=gen))
    cache[3][cache[3] > 1e21] = 1.0  # (blocks of no sequence)
    check_decode(torch.randn((24, 2 * group, d), generator=gen), cache)
    check_decode(torch.randn((24, 2 * group, d), generator=gen).to(torch.bfloat16), cache, out_dtype=torch.float32)


def hidden(gen, lens, hkv, bs, d, code, pattern):
    """A cache in which `pattern` says of each block whether its V scale is around 1e9 instead of 1e-9, and
    whose keys' first element tells the two apart."""
    cache = list(paged(gen, lens, hkv, bs, d, code))
    cache[3] = 1e-9 * (0.2 + torch.rand(cache[3].shape, generator=gen))
    kc = cache[0].float()
    kc[..., 0] = 0
    for s, n in enumerate(lens):
        for i in range(-(-n // bs)):
            b = int(cache[4][s, i])
            cache[2][b] = 0.2
            kc[b, :, :, 1:] *= 0.03 / 0.2 * (1.0 if code == I8 else 127 / 448)
            if pattern(i):
                kc[b, :, :, 0] = -100
                cache[3][b] *= 1e18
    cache[0] = kc.round().to(code) if code == I8 else kc.to(code)
    return cache


PATTERNS = {"first": lambda i: i < 3, "second": lambda i: i == 1, "alternating": lambda i: i % 2 == 0,
            "last": lambda i: i % 16 == 15, "pairs": lambda i: i // 2 % 2 == 1, "of seven": lambda i: i * 5 % 7 < 3}


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("bs,d,group", FORMS)
@pytest.mark.parametrize("pattern", PATTERNS)
def test_large_values_without_weight_hide_nothing(code, bs, d, group, pattern):
    """V scales 2^60 above the others', in tokens whose weights are e^-70: the others' outputs stay whole."""
    gen = torch.Generator().manual_seed(bs * d + group)
    lens = [16 * bs, 5 * bs - 3, 3000, bs]
    cache = hidden(gen, lens, 1, bs, d, code, PATTERNS[pattern])
    q = torch.randn((len(lens), group, d), generator=gen)
    q[..., 0] = 40.0
    if PATTERNS[pattern](0):  # (a context that holds nothing else is left to the other tests)
        lens[3] = cache[5][3] = 0
    check_rows(q, cache)
    check_rows(q.to(torch.bfloat16), cache)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("bs,d,group", [f for f in FORMS if f[2] > 1])
@pytest.mark.parametrize("pattern", PATTERNS)
def test_heads_of_their_own(code, bs, d, group, pattern):
    """Of one kv head's query heads, some see only the large values, the others only the small ones."""
    gen = torch.Generator().manual_seed(bs * d + group + 1)
    lens = [16 * bs, 200, 3000]
    cache = hidden(gen, lens, 1, bs, d, code, PATTERNS[pattern])
    q = torch.randn((len(lens), group, d), generator=gen)
    q[..., 0] = 40.0
    q[:, ::2, 0] = -40.0
    check_rows(q, cache)
    check_rows(q.to(torch.float16), cache)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bs,d,group", [(16, 64, 4), (16, 64, 8), (8, 64, 8), (32, 128, 8), (16, 128, 2)])
@pytest.mark.parametrize("size", [1.0, 0.13, 0.0021, 1e-5])
def test_small_weights_of_small_scales_add_up(code, dtype, bs, d, group, size):
    """One token of weight one, then 8192 of 2^-16 to 2^-18.6 in blocks whose V scales are `size` times its own,
    and an element of V that only they have.  Its error: a weight is off by 2^-22 of itself or 2^-34 of the
    largest (2^-15 of these), a score of 20 by 2^-19, sums of some 64 steps by 2^-17; together below 2^-14.
    (2^-25 of a weight of 2^7 that a scale of 2^-10 of the unit multiplies is 2^-22 of the largest.)"""
    kc, vc, ks, vs, tables, lens = paged(torch.Generator().manual_seed(26), [bs + 8192], 1, bs, d, code)
    first = int(tables[0, 0])
    kc, vc = kc.float().zero_(), vc.float().zero_()
    ks.fill_(1.0), vs.fill_(size)
    vs[first] = 1.0
    kc[first, 0, 0, 0] = 16
    vc[:, :, :, 1] = 64
    vc[first] = 0
    q = torch.zeros((1, group, d))
    q[0, :, 0] = 0.6931 * (1.0 + 0.023 * torch.arange(group))
    q, cache = q.to(dtype), [kc.to(code), vc.to(code), ks, vs, tables, lens]
    got, want = decode(q, cache, scale=1.0), speclib.decode_block_quant(q, *cache, scale=1.0)
    assert ((got - want)[0, :, 1].abs() <= 2.0 ** -14 * want[0, :, 1]).all(), ((got - want) / want)[0, :, 1]
