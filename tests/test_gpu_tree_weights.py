"""Tree attention of fp16 caches whose weights lie far below their maximum: a long
context behind one dominant token."""
import math

import pytest
import torch

from paged_kv_cache_251_gb300 import workloads as wl
from steplib import attention_bound, check_within, paged, tree_oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,d", [(2, 64), (2, 128), (33, 128)])   # 8 rows a kv head, and 132
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("seqs,n,at", [(1, 131072, 0), (1, 131072, 70000), (152, 8192, 0), (152, 8192, 5000)])
def test_mass_behind_a_dominant_token(dtype, t, d, wide, seqs, n, at):
    """One token 27 powers of two above n - 1 others, which hold n / 2^27 of the mass
    between them: V is 0 there and about 1 elsewhere, so the output is that mass.
    One context cut over all SMs, and an uncut one on each.

    Beside the usual bound, a weight carried in fp16 is off by half of its smallest
    step, 2^-25, at most.  Weights are carried with the maximum in use at 2^11 or
    more, and the denominator is at least that maximum's weight: tokens x 2^-36 x max |v|."""
    from paged_kv_cache_251_gb300 import pa
    h, bs = 4, 32
    k, v, tables, lens = paged(21, [n], 1, d, bs, dtype)
    q = torch.zeros((1, t, h, d), dtype=dtype, device="cuda")
    q[..., 0] = 8.0
    q[..., 1] = wl.normal_tensor(5, 3, (1, t, h), dtype=dtype).cuda()
    k[:, :, :, 0] = 0
    v.copy_(1 + v / 16)
    blk, row = int(tables[0, at // bs]), at % bs
    k[blk, 0, row] = 0
    k[blk, 0, row, 0] = 27 * math.log(2) * math.sqrt(d) / 8
    v[blk, 0, row] = 0
    out_dtype = torch.float32 if wide else dtype
    ref, mag, dx = tree_oracle(q, k, v, tables, lens, [t], None, 1 / math.sqrt(d))
    q = q.expand(seqs, t, h, d).contiguous()
    tables, lens = tables.expand(seqs, -1).contiguous(), lens.expand(seqs).contiguous()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(q.shape, dtype=out_dtype, device="cuda")
    pa.pa_decode_tree(out, q, k, v, tables, lens, err_word=err)
    assert err.item() == 0
    bound = attention_bound(ref, mag, dx, dtype, out_dtype, n)
    if dtype == torch.float16:
        bound = bound + n * 2.0 ** -36 * float(v.abs().max())
    check_within(out, ref, bound)
