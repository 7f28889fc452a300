"""CPU checks of the serving-step operators: refusals at the C interface and in
the binding, rotary frequencies, tree masks, block manager truncate / renew."""
import ctypes
import math

import pytest
import torch

from paged_kv_cache_251_gb300 import build as pbuild
from paged_kv_cache_251_gb300 import workloads as wl

INV, UNS, WS, NOBLK = 1, 2, 3, 5
P, I, F, LL, SZ, D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t,
                      ctypes.c_double)


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(str(pbuild.build()))


def caller(fn, types, ok):
    """call(name=value, ...): fn with the arguments `ok` (in order) and some replaced.
    The addresses are made up: a refused call never touches them."""
    fn.restype = I
    fn.argtypes = types

    def call(**over):
        assert set(over) <= set(ok)
        return fn(*[dict(ok, **over)[name] for name in ok])
    return call


def test_rope_refusals(lib):
    call = caller(lib.pa_rope, [P, P, P, P, I, I, I, I, LL, LL, I, I, F, I, P],
                  dict(out=0x1000, x=0x9000, pos=0x2000, fr=0x3000, n=4, h=8, d=128, rot=128, xs=1024, os=1024, inter=0,
                       dir=1, m=1.0, dt=1, st=None))
    assert call(n=0) == 0
    assert call(d=96) == UNS
    for bad in (dict(n=-1), dict(h=0), dict(rot=0), dict(rot=130), dict(rot=3), dict(xs=1023), dict(os=1000),
                dict(dir=0), dict(m=float("nan")), dict(dt=3), dict(out=0), dict(x=0), dict(pos=0), dict(fr=0),
                dict(x=0x9001), dict(out=0x9000, os=2048)):
        assert call(**bad) == INV, bad


def test_rope_append_refusals(lib):
    call = caller(lib.pa_rope_append_kv,
                  [P, P, P, P, P, P, P, P, P, I, I, I, I, I, LL, LL, LL, I, I, I, F, I, P, P],
                  dict(qo=0x1000, q=0x2000, k=0x3000, v=0x4000, pos=0x5000, sl=0x6000, fr=0x7000, kc=0x8000, vc=0x9000,
                       n=4, h=8, hkv=2, d=128, rot=64, qs=1024, ks=256, vs=256, bs=16, nb=10, inter=0, m=1.0, dt=2,
                       err=None, st=None))
    assert call(n=0) == 0
    assert call(d=32) == UNS and call(bs=12) == UNS
    for bad in (dict(hkv=0), dict(nb=0), dict(qs=1000), dict(ks=255), dict(vs=0), dict(kc=0x8008), dict(vc=0),
                dict(sl=0x6004), dict(q=0x2001), dict(v=0), dict(rot=-2), dict(dt=9),
                dict(qo=0x2000, qs=2048)):
        assert call(**bad) == INV, bad


def test_tree_refusals(lib):
    call = caller(lib.pa_decode_tree,
                  [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, P, SZ, P, P],
                  dict(out=0x1000, q=0x2000, k=0x3000, v=0x4000, bt=0x5000, cl=0x6000, dl=None, mask=0x7000, n=4, t=8,
                       h=8, hkv=2, d=128, bs=16, scale=0.1, dt=2, odt=2, m=8, nb=64, ws=None, wsb=0, err=None,
                       st=None))
    assert call(n=0) == 0
    assert call(h=12, hkv=4) == UNS and call(d=96) == UNS and call(bs=24) == UNS
    for bad in (dict(t=0), dict(t=257), dict(n=-1), dict(h=9), dict(hkv=0), dict(q=0), dict(cl=0), dict(k=0x3008),
                dict(mask=0x7004), dict(scale=float("inf")), dict(dt=4), dict(odt=3), dict(nb=0), dict(m=0),
                dict(out=0x1001)):
        assert call(**bad) == INV, bad
    assert call(m=1000) == WS
    assert call(m=1000, ws=0x100, wsb=16) == WS
    assert call(m=1000, ws=0x108, wsb=1 << 40) == INV


def test_tree_workspace_size(lib):
    f = lib.pa_decode_tree_workspace_size
    f.restype, f.argtypes = SZ, [I] * 8
    F32, BF16 = 0, 2
    assert f(4, 8, 8, 2, 128, 16, 8, BF16) == 0                       # contexts of one 128-token tile are never cut
    # two partials (32 rows), a record each, for 16 CTAs
    assert f(4, 8, 8, 2, 128, 16, 9, BF16) == 16 * (2 * 32 * 130 * 4 + 32)
    assert f(64, 16, 32, 8, 128, 16, 512, BF16) == 152 * (2 * 64 * 130 * 4 + 32)
    assert f(4, 64, 32, 8, 128, 16, 8192, BF16) == 152 * (2 * 256 * 130 * 4 + 32)
    assert f(4, 256, 64, 8, 64, 16, 8192, BF16) == 152 * (2 * 256 * 66 * 4 + 32)   # 2048 rows: tiles of 256
    assert f(4, 8, 8, 2, 128, 16, 16, F32) == 0                       # one 256-token partition
    assert f(4, 8, 8, 2, 128, 16, 64, F32) == 4 * 8 * 8 * 4 * 130 * 4
    assert f(4, 0, 8, 2, 128, 16, 64, F32) == 0 and f(4, 8, 9, 2, 128, 16, 64, F32) == 0
    assert f(4, 8, 8, 2, 128, 16, 64, 3) == 0


def test_scored_refusals(lib):
    size = lib.pa_decode_scored_workspace_size
    size.restype, size.argtypes = SZ, [I] * 6
    need = size(4, 8, 128, 16, 8, 0)
    assert need == 4 * 8 * 2 * 4 + 4 * 8 * 8 * 16 * 4
    assert size(4, 8, 100, 16, 8, 0) == 0
    call = caller(lib.pa_decode_scored,
                  [P, P, P, P, P, P, P, P, I, I, I, I, I, F, LL, I, I, I, I, I, P, SZ, P, P],
                  dict(out=0x1000, so=0x8000, si=0x8000, q=0x2000, k=0x3000, v=0x4000, bt=0x5000, cl=0x6000, n=4, h=8,
                       hkv=2, d=128, bs=16, scale=0.1, stride=128, dt=1, odt=0, m=8, nb=64, part=0, ws=0x100000,
                       wsb=need, err=None, st=None))
    assert call(n=0) == 0
    assert call(h=24) == UNS and call(bs=4) == UNS
    for bad in (dict(so=0), dict(so=0x8002), dict(si=0x8001), dict(stride=127), dict(q=0), dict(k=0x3004),
                dict(scale=float("nan")), dict(ws=0x100008), dict(part=40), dict(dt=7)):
        assert call(**bad) == INV, bad
    assert call(wsb=need - 1) == WS and call(ws=None) == WS


def test_select_refusals(lib):
    call = caller(lib.pa_evict_select, [P, P, P, P, P, I, I, I, I, LL, P, P],
                  dict(keep=0x1000, new=0x2000, so=None, s=0x3000, cl=0x4000, n=2, hkv=2, budget=16, recent=4,
                       stride=64, err=None, st=None))
    assert call(n=0) == 0
    for bad in (dict(n=-1), dict(hkv=0), dict(budget=0), dict(recent=-1), dict(recent=17), dict(stride=0),
                dict(keep=0), dict(new=0), dict(s=0), dict(cl=0), dict(s=0x3002), dict(so=0x3001)):
        assert call(**bad) == INV, bad


def test_compact_refusals(lib):
    call = caller(lib.pa_compact_kv, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P, P],
                  dict(k=0x1000, v=0x2000, keep=0x3000, kl=0x4000, bl=None, bt=0x5000, dst=None, n=2, kh=1, ks=8, hkv=4,
                       d=64, bs=8, m=4, dm=0, nb=16, dt=0, err=None, st=None))
    assert call(n=0) == 0 and call(ks=0) == 0
    assert call(d=80) == UNS and call(bs=64) == UNS
    for bad in (dict(kh=2), dict(kh=0), dict(hkv=0), dict(ks=-1), dict(m=0), dict(nb=0), dict(dt=3),
                dict(dst=0x6000), dict(k=0x1004), dict(keep=0), dict(kl=0), dict(bt=0)):
        assert call(**bad) == INV, bad


def test_long_rows_are_refused(lib):
    """Above 2^30 tokens a row: 32-bit positions would not leave room for a tile
    past the end.  At 2^30 the call goes on to its other checks."""
    tree = caller(lib.pa_decode_tree,
                  [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, P, SZ, P, P],
                  dict(out=0x1000, q=0x2000, k=0x3000, v=0x4000, bt=0x5000, cl=0x6000, dl=None, mask=0x7000, n=1, t=8,
                       h=8, hkv=2, d=128, bs=32, scale=0.1, dt=2, odt=2, m=8, nb=64, ws=None, wsb=0, err=None,
                       st=None))
    assert tree(m=1 << 25) == WS and tree(m=(1 << 25) + 1) == UNS and tree(m=(1 << 25) + 1, dt=0, odt=0) == UNS
    scored = caller(lib.pa_decode_scored,
                    [P, P, P, P, P, P, P, P, I, I, I, I, I, F, LL, I, I, I, I, I, P, SZ, P, P],
                    dict(out=0x1000, so=0x8000, si=0x8000, q=0x2000, k=0x3000, v=0x4000, bt=0x5000, cl=0x6000, n=1,
                         h=8, hkv=2, d=128, bs=32, scale=0.1, stride=1 << 31, dt=1, odt=0, m=8, nb=64, part=0, ws=None,
                         wsb=0, err=None, st=None))
    assert scored(m=1 << 25) == WS and scored(m=(1 << 25) + 1) == UNS
    select = caller(lib.pa_evict_select, [P, P, P, P, P, I, I, I, I, LL, P, P],
                    dict(keep=None, new=0x2000, so=None, s=0x3000, cl=0x4000, n=2, hkv=2, budget=16, recent=4,
                         stride=64, err=None, st=None))
    assert select(stride=1 << 30, budget=1 << 30) == INV
    assert select(stride=(1 << 30) + 1) == UNS and select(budget=(1 << 30) + 1) == UNS
    compact = caller(lib.pa_compact_kv, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P, P],
                     dict(k=None, v=0x2000, keep=0x3000, kl=0x4000, bl=None, bt=0x5000, dst=None, n=2, kh=1, ks=8,
                          hkv=4, d=64, bs=8, m=4, dm=0, nb=16, dt=0, err=None, st=None))
    assert compact(ks=1 << 30) == INV and compact(ks=(1 << 30) + 1) == UNS


def test_binding_refusals():
    """The binding refuses what the C interface cannot see: shapes, types, and
    tensors off the GPU."""
    from paged_kv_cache_251_gb300 import pa
    x = torch.zeros((2, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope(x, x, torch.zeros(2, dtype=torch.int32), pa.pa_rope_frequencies(64))
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_evict_select(torch.zeros((1, 1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), None,
                           torch.zeros((1, 1, 8)), torch.zeros(1, dtype=torch.int32), 4, 0)
    with pytest.raises(ValueError, match="scaling"):
        pa.pa_rope_frequencies(64, scaling="cubic")
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_rope_frequencies(63)
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_rope_frequencies(64, scaling="ramp", factor=4)          # no original length
    with pytest.raises(ValueError, match="dense"):
        pa._rows(torch.zeros((3, 64, 4)).transpose(1, 2), "x")
    with pytest.raises(ValueError, match="parent"):
        pa.tree_mask_from_parents(torch.tensor([[-1, 1]]))


def test_rope_frequencies():
    from paged_kv_cache_251_gb300 import pa
    r = 128
    plain = [10000.0 ** (-2 * i / r) for i in range(r // 2)]
    torch.testing.assert_close(pa.pa_rope_frequencies(r), torch.tensor(plain, dtype=torch.float64), rtol=1e-14, atol=0)
    lin = pa.pa_rope_frequencies(r, scaling="linear", factor=4)
    torch.testing.assert_close(lin, torch.tensor(plain, dtype=torch.float64) / 4, rtol=1e-14, atol=0)
    # an enlarged base: the first pair keeps its frequency, the last one is divided by factor
    big = pa.pa_rope_frequencies(r, scaling="base", factor=4)
    assert big[0] == 1 and abs(big[-1] / plain[-1] * 4 - 1) < 1e-12
    # by wavelength: fast pairs keep theirs, slow ones are divided, monotone between
    ramp = pa.pa_rope_frequencies(r, scaling="ramp", factor=8, original_len=8192, low=1, high=4)
    ratio = torch.tensor(plain, dtype=torch.float64) / ramp
    turns = torch.tensor(plain, dtype=torch.float64) * 8192 / (2 * math.pi)
    assert (ratio[turns >= 4] == 1).all()
    torch.testing.assert_close(ratio[turns <= 1], torch.full_like(ratio[turns <= 1], 8.0))
    assert (ratio[1:] >= ratio[:-1] - 1e-12).all() and bool(((ratio > 1.001) & (ratio < 7.9)).any())
    assert pa.pa_rope_frequencies(2, scaling="base", factor=4).tolist() == [1.0]


def test_tree_mask_from_parents():
    from paged_kv_cache_251_gb300 import pa
    t = 130
    parents = torch.full((2, t), -1)
    parents[1] = torch.arange(t) - 1                      # a chain
    m = pa.tree_mask_from_parents(parents)
    assert m.shape == (2, t, 3) and m.dtype == torch.int64
    for i in range(t):
        own = sum((int(m[0, i, w]) & (2 ** 64 - 1)) << (64 * w) for w in range(3))
        chain = sum((int(m[1, i, w]) & (2 ** 64 - 1)) << (64 * w) for w in range(3))
        assert own == 1 << i and chain == (1 << (i + 1)) - 1


def test_block_manager_truncate_and_renew():
    from paged_kv_cache_251_gb300 import pa
    from paged_kv_cache_251_gb300.blocks import BlockManager
    bm = BlockManager(10, 8, 3, 6)
    bm.add_sequence(0)
    bm.extend(0, 30)                                      # blocks 0 .. 3
    bm.fork(0, 1)
    bm.truncate(0, 17)                                    # 3 blocks left; the child still holds the fourth
    tables, lens = bm.tables()
    assert lens.tolist() == [17, 30, 0] and tables[0].tolist() == [0, 1, 2, -1, -1, -1]
    assert [bm.refcount(b) for b in range(4)] == [2, 2, 2, 1] and bm.num_free() == 6
    bm.truncate(0, 16)                                    # a block boundary
    assert bm.refcount(2) == 1 and bm.length(0) == 16
    slots, pairs = bm.append([0])
    assert slots.tolist() == [4 * 8] and pairs.numel() == 0
    for seq, n in ((0, 18), (0, -1), (2, 0), (5, 0)):
        with pytest.raises(pa.PagedAttentionError) as e:
            bm.truncate(seq, n)
        assert e.value.status == INV
    bm.renew(1, 20)                                       # 3 fresh blocks, the old ones dropped
    tables, lens = bm.tables()
    assert lens.tolist() == [17, 20, 0] and tables[1].tolist() == [5, 6, 7, -1, -1, -1]
    assert [bm.refcount(b) for b in range(4)] == [1, 1, 0, 0]
    free = bm.num_free()
    with pytest.raises(pa.PagedAttentionError) as e:
        bm.renew(1, 48)                                   # six blocks, four free
    assert e.value.status == NOBLK and bm.num_free() == free and bm.length(1) == 20
    with pytest.raises(pa.PagedAttentionError):
        bm.renew(1, 49)                                   # more than a table row holds
    bm.truncate(1, 0)
    assert bm.length(1) == 0 and bm.num_free() == free + 3
    bm.add_sequence(2, ring_blocks=2)
    with pytest.raises(pa.PagedAttentionError):
        bm.truncate(2, 0)
    with pytest.raises(pa.PagedAttentionError):
        bm.renew(2, 0)
