"""pa_append_kv_block_quant where two tokens of a call name one slot."""
import pytest
import torch

import speclib
from test_gpu_block_quant import E4M3, I8, append, pool, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("n,dup", [(3, (1, 2)), (512, (0, 300)), (700, (0, 699)), (700, (5, 6)), (700, (17, 400)),
                                   (1300, (1299, 2)), (2000, (800, 803))])
@pytest.mark.parametrize("row", [0, 3, 15])
def test_two_tokens_of_one_slot(code, n, dup, row):
    """The cache is that of a call with one of the two, whole: at a block's row 0, its lowest written row or a
    later one, in one window of tokens or far apart; every other block is as it would be."""
    gen = torch.Generator().manual_seed(n + row)
    nb = n // 8 + 4
    cache = pool(gen, nb, 2, 16, 64, code)
    slots = torch.randperm((nb - 1) * 16, generator=gen)[:n]
    slots[dup[0]] = slots[dup[1]] = (nb - 1) * 16 + row
    more = n - 1 if n - 1 not in dup else n - 3
    if n > 3:
        slots[more] = (nb - 1) * 16 + 15 if row != 15 else (nb - 1) * 16 + 2  # another row of that block
    k, v = rows(gen, n, 2, 64, torch.float32), rows(gen, n, 2, 64, torch.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = append(k, v, slots, *cache, err_word=err)
    assert err.item() == 0
    fits = []
    for j in dup:
        one = slots.clone()
        one[j] = -1
        want = speclib.append_block_quant(k, v, one, *cache)
        fits.append(all(torch.equal(x.cpu().double(), w) for x, w in
                        zip(got, (want[0], want[1], want[2], want[3]))))
    assert any(fits)
