"""pa_append_kv_block_quant where it codes older rows again."""
import pytest
import torch

import speclib
from test_gpu_block_quant import E4M3, append, pool, rows

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
