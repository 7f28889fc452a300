"""Scores of pa_decode_block_quant: as good as fp32 sums of the exact products, whatever the queries' mean."""
import pytest
import torch

import speclib
from test_gpu_block_quant import E4M3, I8, paged
from test_gpu_block_quant_scales import decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bs,d,group", [(16, 128, 4), (16, 128, 8), (8, 64, 2), (32, 64, 8)])
@pytest.mark.parametrize("mean", [0.0, 1.0, 4.0, 16.0])
def test_scores_of_small_codes(code, dtype, bs, d, group, mean):
    """Codes of -1, 0 and 1, in blocks whose scales one large element sets.  A score is off by
    at most 20 * 2^-24 of S = scale * sum |q k|: exact products, d / 16 sums of 16 that may be truncated
    (2^-23 of S each, 8 of them), three roundings by scales and one of the running maximum.  Weights take
    twice that, and 2^-19 for the exponential, the weights' 22 bits and the sums."""
    gen = torch.Generator().manual_seed(50)
    lens = [33, 500, 3000]
    cache = list(paged(gen, lens, 2, bs, d, code))
    kc = torch.randint(-1, 2, cache[0].shape, generator=gen).float()
    kc[:, :, -1, 0] = 127
    q = mean + torch.randn((len(lens), 2 * group, d), generator=gen)
    q[:, :, 0] = 0.25  # (the large element's own score stays in line)
    cache[0] = kc.to(code)
    cache[2].fill_(40.0 * d ** 0.5 / (max(mean, 0.8) * d * 0.667))  # S around 40
    q = q.to(dtype)
    got, want = decode(q, cache), speclib.decode_block_quant(q, *cache)
    size = speclib.decode_block_quant(q, cache[0], torch.ones_like(cache[1].float()).to(code), cache[2],
                                      cache[3] * speclib.QMAX[code], *cache[4:])[..., :1]
    s = d ** -0.5 * q.double().abs().sum(-1, keepdim=True) * cache[2].max().double()  # sum |q k| at most
    s = s + d ** -0.5 * 0.25 * 128 * cache[2].max().double()
    far = (got - want).abs() - size * (2 * 20 * 2.0 ** -24 * s + 2.0 ** -19)
    assert far.max() <= 0, ((got - want).abs() / size).max().item()
