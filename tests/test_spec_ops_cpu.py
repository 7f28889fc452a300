"""CPU checks of the verification, the block-scaled caches and the page tables:
refusals at the C interface and in the binding, workspace sizes."""
import ctypes

import pytest
import torch

from paged_kv_cache_251_gb300 import build as pbuild
from test_step_ops_cpu import INV, UNS, WS, P, I, F, LL, SZ, caller


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(str(pbuild.build()))


def test_verify_refusals(lib):
    call = caller(lib.pa_verify_drafts, [P, P, P, P, P, P, P, P, P, I, I, I, LL, LL, I, P, P],
                  dict(al=0x1000, ac=0x2000, tk=0x3000, tp=0x4000, dp=0x5000, dt=0x6000, dl=0x7000, pa=0x8000, u=0x9000,
                       n=2, t=4, v=100, ts=100, ds=100, ty=0, err=None, st=None))
    assert call(n=0) == 0
    assert call(v=(1 << 30) + 1, ts=1 << 31, ds=1 << 31) == UNS and call(n=1 << 28) == UNS
    for bad in (dict(n=-1), dict(t=0), dict(t=257), dict(v=0), dict(ts=99), dict(ds=99), dict(ty=3), dict(al=0),
                dict(ac=0), dict(tk=0), dict(tp=0), dict(dt=0), dict(u=0), dict(tp=0x4002), dict(ty=1, dp=0x5001),
                dict(tk=0x3002), dict(u=0x9001), dict(pa=0x8002), dict(dl=0x7001), dict(err=0x1002)):
        assert call(**bad) == INV, bad


def test_append_refusals(lib):
    call = caller(lib.pa_append_kv_block_quant, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, SZ, P, P],
                  dict(k=0x1000, v=0x2000, sl=0x3000, kc=0x4000, vc=0x5000, ks=0x6000, vs=0x7000, n=4, hkv=2, d=128,
                       bs=16, nb=10, dt=1, cdt=3, ws=0, wsb=0, err=None, st=None))
    assert call(n=0) == 0
    assert call(d=96) == UNS and call(bs=12) == UNS
    assert call(n=513) == WS and call(n=513, ws=0x8000, wsb=683) == WS
    for bad in (dict(n=-1), dict(hkv=0), dict(nb=0), dict(dt=3), dict(cdt=1), dict(k=0), dict(v=0x2008), dict(sl=0x3004),
                dict(kc=0x4008), dict(vc=0), dict(ks=0x6002), dict(vs=0), dict(ws=0x8002), dict(err=0x1001)):
        assert call(**bad) == INV, bad
    size = lib.pa_append_kv_block_quant_workspace_size
    size.restype, size.argtypes = SZ, [I, I, I]
    assert size(512, 16, 10) == 0 and size(513, 16, 10) == 684 and size(513, 12, 10) == 0 and size(513, 16, 0) == 0
    assert size(600, 32, 1 << 30) == (4 << 35) + 4 * 601
    assert call(n=(1 << 30) + 1) == UNS and call(hkv=(1 << 29) + 1) == UNS


def test_decode_refusals(lib):
    size = lib.pa_decode_block_quant_workspace_size
    size.restype, size.argtypes = SZ, [I] * 6
    need = size(4, 8, 2, 128, 16, 8)
    assert need > 0 and size(4, 8, 3, 128, 16, 8) == 0 and size(4, 8, 2, 96, 16, 8) == 0 and size(0, 8, 2, 128, 16, 8) == 0
    assert size(4, 8, 2, 128, 16, 1 << 27) == 0
    call = caller(lib.pa_decode_block_quant, [P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, I, I, I, I, I, P, SZ, P, P],
                  dict(out=0x1000, q=0x2000, kc=0x3000, vc=0x4000, ks=0x5000, vs=0x6000, bt=0x7000, cl=0x8000, n=4, h=8,
                       hkv=2, d=128, bs=16, sc=0.1, w=0, dt=1, cdt=4, odt=0, m=8, nb=64, ws=0x10000, wsb=need, err=None,
                       st=None))
    assert call(n=0) == 0
    assert call(d=96) == UNS and call(bs=12) == UNS and call(h=12, hkv=4) == UNS and call(m=1 << 27) == UNS
    assert call(ws=0) == WS and call(wsb=need - 1) == WS
    for bad in (dict(n=-1), dict(h=9), dict(h=0), dict(hkv=0), dict(w=-1), dict(m=0), dict(nb=0), dict(dt=3), dict(cdt=2),
                dict(odt=4), dict(sc=float("nan")), dict(q=0), dict(kc=0x3008), dict(vc=0), dict(ks=0), dict(vs=0x6002),
                dict(bt=0), dict(cl=0x8001), dict(out=0x1002), dict(ws=0x10008), dict(err=0x1002)):
        assert call(**bad) == INV, bad


def test_pages_refusals(lib):
    size = lib.pa_pages_workspace_size
    size.restype, size.argtypes = SZ, [I, I]
    assert size(4, 100) == 16 * 104 and size(-1, 100) == 0 and size(4, 0) == 0
    call = caller(lib.pa_pages_update, [P] * 10 + [I] * 5 + [P, SZ, P, P],
                  dict(nt=0x1000, nr=0x2000, pr=0x3000, st=0x4000, t=0x9000, r=0x5000, ln=0x6000, pa=0x7000, k=0x8000,
                       g=0x8800, n=4, o=4, m=8, bs=16, nb=100, ws=0x10000, wsb=1664, err=None, stream=None))
    assert call(ws=0) == WS and call(wsb=1663) == WS and call(o=5) == WS
    assert call(m=1 << 27) == UNS and call(bs=1, m=1 << 21) == UNS  # (needs are summed in 32 bits)
    for bad in (dict(n=-1), dict(o=-1), dict(m=0), dict(bs=0), dict(nb=0), dict(nt=0), dict(nr=0), dict(pr=0),
                dict(st=0), dict(t=0), dict(r=0), dict(ln=0), dict(k=0), dict(g=0), dict(pa=0, n=5, wsb=1 << 20),
                dict(pr=0x3004), dict(nt=0x1002), dict(ws=0x10002), dict(t=0x1000), dict(t=0x1010), dict(nt=0x9070),
                dict(nr=0x5010), dict(err=0x1)):
        assert call(**bad) == INV, bad
    call = caller(lib.pa_pages_compact, [P] * 8 + [I] * 5 + [P, SZ, P, P],
                  dict(nt=0x1000, nr=0x2000, rm=0x2800, pr=0x3000, st=0x4000, t=0x9000, r=0x5000, ln=0x6000, n=4, m=8,
                       bs=16, nb=100, mv=50, ws=0x10000, wsb=1664, err=None, stream=None))
    assert call(ws=0) == WS and call(wsb=1663) == WS
    assert call(bs=1, m=1 << 21) == UNS and call(mv=(1 << 30) + 1) == UNS and call(n=(1 << 30) + 1) == UNS
    for bad in (dict(n=-1), dict(m=0), dict(bs=-1), dict(nb=0), dict(mv=-1), dict(nt=0), dict(nr=0), dict(rm=0),
                dict(pr=0), dict(st=0), dict(t=0), dict(r=0), dict(ln=0), dict(pr=0x3004), dict(rm=0x2801),
                dict(nt=0x9010), dict(nr=0x5004), dict(err=0x3)):
        assert call(**bad) == INV, bad


def test_copy_pages_refusals(lib):
    fn = lib.pa_copy_pages
    fn.restype, fn.argtypes = I, [P, I, P, P, I, I, P, P]

    def call(pairs=0x1000, n=3, pools=(0x2000, 0x3000), sizes=(64, 4), k=None, nb=10, err=None):
        at, size = (ctypes.c_void_p * len(pools))(*pools), (LL * len(sizes))(*sizes)
        return fn(pairs, n, at, size, len(pools) if k is None else k, nb, err, None)

    assert call(n=0) == 0
    assert call(sizes=(1 << 62, 4)) == UNS and call(n=(1 << 30) + 1) == UNS
    for bad in (dict(n=-1), dict(nb=0), dict(k=0), dict(k=9), dict(pairs=0), dict(pairs=0x1004), dict(pools=(0x2000, 0)),
                dict(pools=(0x2002, 0x3000)), dict(sizes=(6, 4)), dict(sizes=(0, 4)), dict(sizes=(-4, 4)), dict(err=0x1)):
        assert call(**bad) == INV, bad


# ---------------------------------------------------------------------------
# The binding, with tensors on the CPU: its checks come before any address is used


def test_binding_refuses_cpu_tensors():
    from paged_kv_cache_251_gb300 import pa
    z = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_verify_drafts(z[:, 0], z, z, torch.zeros(2, 4, 9), z, torch.zeros(2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_pages_update(z, z[0], z, z, z, z[0], z[:, 0], z[:, 0], z[:, 0], 16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_copy_pages(torch.zeros(2, 2, dtype=torch.int64), [z])


class _Fake:
    """The checks see CPU tensors as if they were on device 0."""

    def __init__(self, monkeypatch, pa):
        self.calls = []
        monkeypatch.setattr(pa, "_dense", lambda first, *rest: 0)
        monkeypatch.setattr(pa, "_call", lambda fn, dev, stream, *args: self.calls.append(args))
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)


def test_binding_checks_of_verify(monkeypatch):
    from paged_kv_cache_251_gb300 import pa
    fake = _Fake(monkeypatch, pa)
    i32 = dict(dtype=torch.int32)

    def call(t=3, **over):
        a = dict(accept_lens=torch.zeros(2, **i32), accepted=torch.zeros(2, t, **i32), tokens=torch.zeros(2, t + 1, **i32),
                 target_probs=torch.zeros(2, t + 1, 9), draft_tokens=torch.zeros(2, t, **i32),
                 uniforms=torch.zeros(2, t + 1), draft_probs=torch.zeros(2, t, 9))
        pa.pa_verify_drafts(**dict(a, **over))
        return fake.calls[-1]

    assert call()[9:15] == (2, 3, 9, 9, 9, 0)
    wide = torch.zeros(2, 4, 12)[:, :, :9]
    assert call(target_probs=wide)[12] == 12
    assert call(draft_probs=None)[13] == 0
    assert call(t=1, target_probs=torch.zeros(2, 2, 9), draft_probs=torch.zeros(2, 1, 11)[:, :, :9])[13] == 11
    for bad in (dict(accepted=torch.zeros(2, 4, **i32)), dict(tokens=torch.zeros(2, 3, **i32)),
                dict(target_probs=torch.zeros(2, 3, 9)), dict(uniforms=torch.zeros(2, 3)),
                dict(draft_probs=torch.zeros(2, 3, 8)), dict(draft_probs=torch.zeros(2, 3, 9, dtype=torch.float16)),
                dict(draft_lens=torch.zeros(3, **i32)), dict(parents=torch.zeros(2, 2, **i32)),
                dict(target_probs=torch.zeros(2, 4, 18)[:, :, ::2]), dict(target_probs=torch.zeros(2, 9, 9)[:, ::2][:, :4]),
                dict(target_probs=torch.zeros(1, 4, 9).expand(2, 4, 9))):
        if "target_probs" in bad and bad["target_probs"].stride() == (81, 18, 1):
            with pytest.raises(ValueError):
                call(**bad)
            continue
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    for bad in (dict(draft_tokens=torch.zeros(2, 3, dtype=torch.int64)), dict(uniforms=torch.zeros(2, 4).double()),
                dict(target_probs=torch.zeros(2, 4, 9).double(), draft_probs=None), dict(parents=torch.zeros(2, 3))):
        with pytest.raises(TypeError):
            call(**bad)


def test_binding_checks_of_block_quant(monkeypatch):
    from paged_kv_cache_251_gb300 import pa
    fake = _Fake(monkeypatch, pa)

    def pool(dtype=torch.int8, shape=(5, 2, 16, 64)):
        return torch.zeros(shape).to(dtype)

    def append(**over):
        a = dict(k=torch.zeros(3, 2, 64), v=torch.zeros(3, 2, 64), slot_mapping=torch.zeros(3, dtype=torch.int64),
                 k_cache=pool(), v_cache=pool(), k_scales=torch.zeros(5, 2), v_scales=torch.zeros(5, 2))
        pa.pa_append_kv_block_quant(**dict(a, **over))
        return fake.calls[-1]

    assert append()[7:14] == (3, 2, 64, 16, 5, 0, 3)
    for bad in (dict(k=torch.zeros(3, 2, 128)), dict(v=torch.zeros(2, 2, 64)), dict(v_cache=pool(torch.float8_e4m3fn)),
                dict(v_cache=pool(shape=(5, 2, 16, 128))), dict(k_cache=pool(torch.float16)), dict(k_scales=torch.zeros(5, 1)),
                dict(v_scales=torch.zeros(5, 2).half()), dict(slot_mapping=torch.zeros(3, dtype=torch.int32)),
                dict(k=torch.zeros(3, 2, 64).half())):
        with pytest.raises((ValueError, TypeError)):
            append(**bad)

    def decode(**over):
        a = dict(out=torch.zeros(3, 8, 64), q=torch.zeros(3, 8, 64), k_cache=pool(), v_cache=pool(),
                 k_scales=torch.zeros(5, 2), v_scales=torch.zeros(5, 2),
                 block_tables=torch.zeros(3, 4, dtype=torch.int32), context_lens=torch.zeros(3, dtype=torch.int32))
        pa.pa_decode_block_quant(**dict(a, **over))
        return fake.calls[-1]

    assert decode()[8:13] == (3, 8, 2, 64, 16)
    for bad in (dict(out=torch.zeros(3, 8, 128)), dict(q=torch.zeros(3, 8, 128)), dict(context_lens=torch.zeros(3)),
                dict(block_tables=torch.zeros(2, 4, dtype=torch.int32)), dict(k_scales=torch.zeros(4, 2)),
                dict(context_lens=torch.zeros(4, dtype=torch.int32)), dict(q=torch.zeros(3, 8, 64).double())):
        with pytest.raises((ValueError, TypeError)):
            decode(**bad)


def test_binding_checks_of_pages(monkeypatch):
    from paged_kv_cache_251_gb300 import pa
    fake = _Fake(monkeypatch, pa)

    def i32(*s):
        return torch.zeros(s, dtype=torch.int32)

    def update(**over):
        a = dict(new_tables=i32(3, 4), new_ref_counts=i32(9), pairs=torch.zeros(3, 2, dtype=torch.int64), status=i32(4),
                 tables=i32(2, 4), ref_counts=i32(9), lens=i32(2), keep_lens=i32(3), grow_lens=i32(3), block_size=16,
                 parents=i32(3))
        pa.pa_pages_update(**dict(a, **over))
        return fake.calls[-1]

    assert update()[10:15] == (3, 2, 4, 16, 9)
    for bad in (dict(new_tables=i32(3, 5)), dict(new_ref_counts=i32(8)), dict(pairs=i32(3, 2)), dict(status=i32(3)),
                dict(lens=i32(3)), dict(keep_lens=i32(2)), dict(grow_lens=i32(4)), dict(parents=i32(2)),
                dict(pairs=torch.zeros(2, 2, dtype=torch.int64)), dict(tables=torch.zeros(2, 4))):
        with pytest.raises((ValueError, TypeError)):
            update(**bad)

    def compact(**over):
        a = dict(new_tables=i32(2, 4), new_ref_counts=i32(9), remap=i32(9), pairs=torch.zeros(5, 2, dtype=torch.int64),
                 status=i32(4), tables=i32(2, 4), ref_counts=i32(9), lens=i32(2), block_size=16)
        pa.pa_pages_compact(**dict(a, **over))
        return fake.calls[-1]

    assert compact()[8:13] == (2, 4, 16, 9, 5)
    for bad in (dict(new_tables=i32(3, 4)), dict(remap=i32(8)), dict(remap=torch.zeros(9)), dict(lens=i32(3))):
        with pytest.raises((ValueError, TypeError)):
            compact(**bad)
    pairs = torch.zeros(5, 2, dtype=torch.int64)
    pa.pa_copy_pages(pairs, [torch.zeros(7, 3, 4), torch.zeros(7)])
    assert fake.calls[-1][1] == 5 and list(fake.calls[-1][3]) == [48, 4] and fake.calls[-1][4:6] == (2, 7)
    for bad in ((pairs.int(), [torch.zeros(7)]), (pairs, []), (pairs, [torch.zeros(7), torch.zeros(6)]),
                (torch.zeros(5, 3, dtype=torch.int64), [torch.zeros(7)])):
        with pytest.raises((ValueError, TypeError)):
            pa.pa_copy_pages(*bad)
