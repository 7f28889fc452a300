"""Rotation angles of far positions against exact arithmetic."""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu

# 1 / (2 pi) to 60 digits
PER_RADIAN = Fraction("0.159154943091895335768883763372514362034459645740456448747667")


@pytest.mark.parametrize("pos", [2 ** 31 - 1, -(2 ** 31), 1999999973, -1000003, 4097, 1])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("inverse", [False, True])
def test_small_angles_of_far_positions(pos, sign, inverse):
    """Frequencies for which position * freq is a whole number of turns and little
    more: the sine is that little, so an error of the angle stands alone.

    The angle is within 2^-31 turn; then roundings relative to it: its conversion to
    fp32, sincospi (2 u) and the product with 1 (exact), 4 u in all with room."""
    from paged_kv_cache_251_gb300 import pa
    whole = [0, 1, 2, 3, 17, 1000, 4095, 123457, 1999999, 99999989, 268435399, 1 << 28]
    freqs, turns = [], []
    for i, k in enumerate(whole * 2):
        k = k if abs(pos) > 2 * k else 0
        f = sign * (2 * math.pi * k + (1e-4 if i < len(whole) else -3e-3)) / abs(pos)
        freqs.append(f)
        t = Fraction(f) * pos * (-1 if inverse else 1) * PER_RADIAN
        turns.append(float(t - round(t)))              # a small remainder, exact to 53 bits
    n = len(freqs)
    x = torch.zeros((1, 1, 64), device="cuda")
    x[..., :n] = 1.0
    out = pa.pa_rope(torch.empty_like(x), x, torch.tensor([pos], dtype=torch.int32, device="cuda"),
                     torch.tensor(freqs, dtype=torch.float64, device="cuda"), inverse=inverse)
    want = torch.sin(2 * math.pi * torch.tensor(turns, dtype=torch.float64))
    got = out[0, 0, n:2 * n].double().cpu()
    assert float(want.abs().max()) < 4e-3
    over = (got - want).abs() - (2 * math.pi * 2.0 ** -31 + want.abs() * 4 * 2.0 ** -24)
    assert float(over.max()) <= 0, f"{float((got - want).abs().max()):.3e} off"
    assert ((out[0, 0, :n].double().cpu() - torch.cos(2 * math.pi * torch.tensor(turns))).abs() <= 2.0 ** -23).all()


def test_frequencies_of_the_schemes():
    """Every frequency of the plain and the ramped scheme at positions near both ends,
    against the exact fraction of a turn."""
    from paged_kv_cache_251_gb300 import pa
    pos = [2 ** 31 - 1, 2 ** 31 - 12345, -(2 ** 31), 10 ** 9 + 7, 131071]
    for scheme in (dict(), dict(scaling="ramp", factor=8, original_len=8192)):
        freqs = pa.pa_rope_frequencies(128, **scheme)
        x = torch.zeros((len(pos), 1, 128), device="cuda")
        x[..., :64] = 1.0
        out = pa.pa_rope(torch.empty_like(x), x, torch.tensor(pos, dtype=torch.int32, device="cuda"), freqs.cuda())
        for i, p in enumerate(pos):
            t = [Fraction(f) * p * PER_RADIAN for f in freqs.tolist()]
            a = 2 * math.pi * torch.tensor([float(u - round(u)) for u in t], dtype=torch.float64)
            # the fraction in half turns rounded to fp32 (2^-25 of one, at most), sincospi 2 u, 2^-31 turn
            bound = math.pi * 2.0 ** -25 + 2 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -31
            assert ((out[i, 0, 64:].double().cpu() - torch.sin(a)).abs() <= bound).all()
            assert ((out[i, 0, :64].double().cpu() - torch.cos(a)).abs() <= bound).all()
