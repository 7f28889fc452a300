"""GPU parity of pa_rope and pa_rope_append_kv against the rotation in 64 bits."""
import math

import pytest
import torch

from paged_kv_cache_251_gb300 import workloads as wl
from steplib import U32, half_step

pytestmark = pytest.mark.gpu


def rotate64(x, positions, freqs, rot, interleaved, mscale, sign=1):
    """The rotation in float64, and |x_a| + |x_b| per rotated element (0 past rot)."""
    x = x.double()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    ang = sign * positions.double()[:, None, None] * freqs.to(x.device)
    c, s = torch.cos(ang) * mscale, torch.sin(ang) * mscale
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def check(got, ref, mag, mscale, max_angle):
    """Cosine and sine: the angle's fp32 rounding is pi u, sincospi 2 u, the
    scaling u; the products and the sum 1.5 u more; freq / 2 pi in double is
    off by 2^-52 relative, times the angle; then the output's own rounding."""
    inner = mag * abs(mscale) * (8 * U32 + max_angle * 2.0 ** -51)
    bound = inner + half_step(got.dtype) * (ref.abs() + inner)
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a step of the subnormals
    over = (got.double() - ref).abs() - bound
    assert float(over.max()) <= 0, f"{float(over.max()):.3e} over the bound"


CASES = [
    # tokens, heads, kv heads, d, rot, interleaved, block
    (1, 1, 1, 64, 64, False, 8),
    (3, 4, 4, 64, 2, True, 16),
    (17, 8, 2, 128, 128, False, 16),
    (300, 32, 8, 128, 64, True, 16),
    (129, 5, 5, 128, 122, False, 32),      # halves off the 16-byte boundary
    (64, 40, 40, 128, 96, True, 8),
    (2500, 2, 1, 64, 32, False, 32),       # several tokens a CTA, a ragged last one
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("sliced", [False, True])
def test_rope_append(case, dtype, sliced):
    from paged_kv_cache_251_gb300 import pa
    n, h, hkv, d, rot, inter, bs = case
    qkv = wl.normal_tensor(n + rot, 3, (n, (h + 2 * hkv) * d), dtype=dtype).cuda()
    q, k, v = (qkv[:, :h * d].view(n, h, d), qkv[:, h * d:(h + hkv) * d].view(n, hkv, d),
               qkv[:, (h + hkv) * d:].view(n, hkv, d))
    if not sliced:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    freqs = pa.pa_rope_frequencies(rot, scaling="ramp", factor=8, original_len=4096)
    pos = wl.randint(7, 1, n, 0, 4000000).to(torch.int32).cuda()
    nb = (n + bs - 1) // bs + 2
    slots = wl.permutation(5, 2, nb * bs)[:n].clone()
    if n > 2:
        slots[1] = -1                      # padding: rotated, not appended
    slots = slots.cuda()
    kc = wl.normal_tensor(1, 4, (nb, hkv, bs, d), dtype=dtype).cuda()
    vc = wl.normal_tensor(1, 5, (nb, hkv, bs, d), dtype=dtype).cuda()
    k0, v0 = kc.clone(), vc.clone()
    out = torch.full((n, h, d), float("nan"), dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_rope_append_kv(out, q, k, v, pos, slots, freqs.cuda(), kc, vc, interleaved=inter, mscale=1.25,
                         err_word=err)
    assert err.item() == 0
    ref, mag = rotate64(q, pos, freqs, rot, inter, 1.25)
    check(out, ref, mag, 1.25, 4e6)
    kref, kmag = rotate64(k, pos, freqs, rot, inter, 1.25)
    good = slots >= 0
    rows_k = kc.transpose(1, 2).reshape(nb * bs, hkv, d)
    rows_v = vc.transpose(1, 2).reshape(nb * bs, hkv, d)
    check(rows_k[slots[good]], kref[good], kmag[good], 1.25, 4e6)
    assert torch.equal(rows_v[slots[good]], v[good])
    # every other row is left as it was
    rest = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    rest[slots[good]] = False
    assert torch.equal(rows_k[rest], k0.transpose(1, 2).reshape(nb * bs, hkv, d)[rest])
    assert torch.equal(rows_v[rest], v0.transpose(1, 2).reshape(nb * bs, hkv, d)[rest])
    # elements past rot pass through bit for bit
    assert torch.equal(out[..., rot:], q[..., rot:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_rows_in_place_and_back(dtype, inter):
    """In place equals out of place; turning back with the direction reversed is
    the transposed rotation: <R x, y> = <x, R^T y>."""
    from paged_kv_cache_251_gb300 import pa
    n, h, d, rot = 37, 6, 128, 64
    x = wl.normal_tensor(2, 3, (n, h, d), dtype=dtype).cuda()
    g = wl.normal_tensor(3, 3, (n, h, d), dtype=dtype).cuda()
    freqs = pa.pa_rope_frequencies(rot, scaling="base", factor=4)
    pos = wl.randint(9, 1, n, -1000, 100000).to(torch.int32).cuda()
    f = freqs.cuda()
    y = pa.pa_rope(torch.empty_like(x), x, pos, f, interleaved=inter, mscale=0.75)
    z = x.clone()
    pa.pa_rope(z, z, pos, f, interleaved=inter, mscale=0.75)
    assert torch.equal(y, z)
    ref, mag = rotate64(x, pos, freqs, rot, inter, 0.75)
    check(y, ref, mag, 0.75, 1e5)
    gx = pa.pa_rope(torch.empty_like(g), g, pos, f, interleaved=inter, inverse=True, mscale=0.75)
    gref, gmag = rotate64(g, pos, freqs, rot, inter, 0.75, sign=-1)
    check(gx, gref, gmag, 0.75, 1e5)
    # the transpose, in 64 bits: <R x, g> = <x, R^T g>
    assert abs(float((ref * g.double()).sum() - (x.double() * gref).sum())) < 1e-9 * float((ref * g).abs().sum())
    # and by differences: d <R x, g> / dx along a direction (the map is linear, so the difference is exact)
    dxn = wl.normal_tensor(4, 3, (n, h, d), dtype=dtype).cuda()
    r2, _ = rotate64(x.double() + 0.5 * dxn.double(), pos, freqs, rot, inter, 0.75)
    slope = ((r2 - ref) * g.double()).sum() / 0.5
    want = (gx.double() * dxn.double()).sum()
    slack = float(((half_step(dtype) * gref.abs() + gmag * 1e-6) * dxn.double().abs()).sum()) + 1e-6
    assert abs(float(slope - want)) <= slack


def test_positions_at_the_end_of_their_range():
    """Angles of positions near 2^31 against integer arithmetic: the fraction of
    a turn of position * freq, exactly, for frequencies that are whole fractions
    of a turn (freq / 2 pi = 1 / m up to the double's rounding)."""
    from paged_kv_cache_251_gb300 import pa
    ms = torch.tensor([7, 1000, 12345, 99991], dtype=torch.int64)
    freqs = 2 * math.pi / ms.double()
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 64, -(2 ** 31), 1999999973], dtype=torch.int64)
    x = torch.zeros((4, 1, 64))
    x[..., :4] = 1.0                                   # x_a = 1, x_b = 0: y = (cos, sin)
    out = pa.pa_rope(torch.empty_like(x).cuda(), x.cuda(), pos.to(torch.int32).cuda(), freqs.cuda()).cpu().double()
    turns = (pos[:, None] % ms).double() / ms.double()
    # the double frequency is off by 2^-53 relative, its product with 1 / 2 pi by 2^-52 more
    tol = 2.0 ** 31 / ms.double() * 2 * math.pi * 2.0 ** -51 + 8 * U32
    assert ((out[:, 0, :4] - torch.cos(2 * math.pi * turns)).abs() <= tol).all()
    assert ((out[:, 0, 4:8] - torch.sin(2 * math.pi * turns)).abs() <= tol).all()


def test_bad_slots_are_flagged_and_skipped():
    from paged_kv_cache_251_gb300 import pa
    n, h, d, bs, nb = 5, 2, 64, 16, 2
    q = torch.randn((n, h, d), device="cuda")
    kc, vc = torch.zeros((nb, h, bs, d), device="cuda"), torch.zeros((nb, h, bs, d), device="cuda")
    slots = torch.tensor([0, nb * bs, -1, 2 ** 40, nb * bs - 1], device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    f = pa.pa_rope_frequencies(d).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    pa.pa_rope_append_kv(out, q, q, q, pos, slots, f, kc, vc, err_word=err)
    assert err.item() == pa.DEVERR_BAD_SLOT
    assert torch.isfinite(out).all()
    assert torch.equal(vc[0, :, 0], q[0]) and torch.equal(vc[1, :, bs - 1], q[4])
    assert int((vc != 0).any(-1).sum()) == 2 * h


def test_misaligned_rows_and_other_stream():
    """Rows that start off a 16-byte boundary, on another stream than the current one."""
    from paged_kv_cache_251_gb300 import pa
    n, h, d = 33, 3, 64
    flat = torch.randn(n * (h * d + 3) + 1, device="cuda").to(torch.bfloat16)
    x = flat[1:].view(n, h * d + 3)[:, :h * d].unflatten(1, (h, d))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freqs = pa.pa_rope_frequencies(d)
    out = torch.empty((n, h, d), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    f = freqs.cuda()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_rope(out, x, pos, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ref, mag = rotate64(x, pos, freqs, d, False, 1.0)
    check(out, ref, mag, 1.0, 100)
