"""Pools beyond what a tensor map addresses are refused by the serving-step decodes."""
import ctypes

import pytest

from paged_kv_cache_251_gb300 import build as pbuild
from test_step_ops_cpu import F, I, LL, P, SZ, UNS, WS, caller


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(str(pbuild.build()))


def test_tree_pools(lib):
    """Above 2^31 - 1 (block, kv head) tiles a 16-bit cache is refused; below, and in
    fp32, a workspace of the queried size is what the call asks for."""
    size = lib.pa_decode_tree_workspace_size
    size.restype, size.argtypes = SZ, [I] * 8
    call = caller(lib.pa_decode_tree,
                  [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, P, SZ, P, P],
                  dict(out=0x1000, q=0x2000, k=0x3000, v=0x4000, bt=0x5000, cl=0x6000, dl=None, mask=0x7000, n=3, t=8,
                       h=8, hkv=2, d=128, bs=16, scale=0.1, dt=2, odt=2, m=4096, nb=64, ws=0x8000, wsb=0, err=None,
                       st=None))
    for dt in (0, 1, 2):
        need = size(3, 8, 8, 2, 128, 16, 4096, dt)
        assert need > 0 and call(dt=dt, odt=dt, wsb=need - 1) == WS and call(dt=dt, odt=dt, ws=None, wsb=need) == WS
        assert call(dt=dt, odt=dt, nb=(1 << 30) - 1, wsb=need - 1) == WS
        assert call(dt=dt, odt=dt, nb=1 << 30, wsb=need - 1) == (UNS if dt else WS)


def test_scored_pools(lib):
    """The scored decode takes pools of up to 2^31 - 1 tiles and as many rows, in every
    type: the kernels without a tensor map would only serve larger ones."""
    call = caller(lib.pa_decode_scored,
                  [P, P, P, P, P, P, P, P, I, I, I, I, I, F, LL, I, I, I, I, I, P, SZ, P, P],
                  dict(out=0x1000, so=0x8000, si=0x8000, q=0x2000, k=0x3000, v=0x4000, bt=0x5000, cl=0x6000, n=4, h=8,
                       hkv=2, d=128, bs=16, scale=0.1, stride=128, dt=1, odt=0, m=8, nb=64, part=0, ws=None, wsb=0,
                       err=None, st=None))
    for dt in (0, 1, 2):
        for h in (2, 8):
            assert call(dt=dt, h=h, nb=(1 << 30) - 1) == WS
            assert call(dt=dt, h=h, nb=1 << 30) == UNS
    assert call(n=1 << 28) == UNS and call(n=(1 << 28) - 1) == WS
