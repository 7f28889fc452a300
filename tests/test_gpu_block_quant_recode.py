"""pa_append_kv_block_quant where it codes older rows again."""
import pytest
import torch

import speclib
from paged_kv_cache_251_gb300 import pa
from test_gpu_block_quant import E4M3, I8, append, pool, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 20, 600])
@pytest.mark.parametrize("bs,d", [(8, 64), (16, 128), (32, 128)])
def test_nan_codes_end_where_a_block_is_coded_again(n, bs, d):
    """A pool of any contents: E4M3 NaN codes of both signs in rows that the call does not write."""
    gen = torch.Generator().manual_seed(n + bs)
    nb = 2 * n + 2
    cache = pool(gen, nb, 2, bs, d, E4M3)
    for codes in cache[:2]:
        raw = codes.view(torch.uint8)
        raw[torch.rand(raw.shape, generator=gen) < 0.3] = 0x7f
        raw[torch.rand(raw.shape, generator=gen) < 0.1] = 0xff
    cache[2][::5] = 0
    slots = torch.randperm(nb, generator=gen)[:n] * bs + torch.randint(1, bs, (n,), generator=gen)
    k, v = (rows(gen, n, 2, d, torch.bfloat16) * 30 for _ in range(2))
    got = append(k, v, slots, *cache)
    want = speclib.append_block_quant(k, v, slots, *cache)
    b = slots // bs
    grew = [want[i + 2][b] > cache[i + 2][b].double() for i in (0, 1)]
    assert all(g.any() for g in grew)
    for x, w in zip(got[2:], want[2:]):
        assert torch.equal(x.cpu().double(), w)
    for x, w, g in zip(got[:2], want[:2], grew):
        assert torch.equal(x.cpu().double()[b][g], w[b][g]) and not w[b][g].isnan().any()


@pytest.mark.parametrize("code", [I8, E4M3])
def test_rejected_drafts_leave_their_scale(code):
    """Steps of one kept token and three drafts that are rejected and written over.  A kept element is off
    by half a step of the scale that it was first stored with, and half a step more of every scale that a
    later token, kept or not, has raised its block to: s / 2 (INT8), the larger of 2^-4 of the element and
    2^-10 s (E4M3)."""
    gen = torch.Generator().manual_seed(60)
    hkv, d, bs = 2, 64, 16
    cache = [x.cuda() for x in pool(gen, 2, hkv, bs, d, code)]
    kept = rows(gen, bs, hkv, d, torch.float32)
    bound = torch.zeros((bs, hkv, d), dtype=torch.float64)
    before = torch.zeros(hkv, dtype=torch.float64)
    for step in range(bs):
        n = min(4, bs - step)
        drafts = rows(gen, n, hkv, d, torch.float32, 1.5)  # (larger than what is kept, often)
        drafts[0] = kept[step]
        pa.pa_append_kv_block_quant(drafts.cuda(), drafts.cuda(), (bs + step + torch.arange(n)).cuda(), *cache)
        scale = cache[2][1].cpu().double()
        raised = scale > before if step else torch.ones(hkv, dtype=torch.bool)
        half = (scale / 2)[:, None].expand(hkv, d)
        for r in range(step + 1):
            size = kept[r].double().abs() + bound[r]
            off = half if code == I8 else torch.maximum(size * 2.0 ** -4, half * 2.0 ** -9)
            bound[r] += torch.where((raised | (r == step))[:, None], off, torch.zeros_like(off))
        before = scale
        value = cache[0][1].cpu().double().transpose(0, 1) * scale[:, None]  # [bs, hkv, d]
        far = (value - kept.double())[:step + 1].abs() - bound[:step + 1] * (1 + 2.0 ** -18)
        assert far.max() <= 0
