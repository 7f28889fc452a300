"""The workspaces that the block-scaled and page calls make for themselves belong to
the call's stream; the calls go to the stream and device that they are given."""
import contextlib
import types

import pytest
import torch

import paged_kv_cache_251_gb300.pa as pa

CALLS = {}


def case(fn):
    CALLS[fn.__name__] = fn
    return fn


@case
def append(dev):
    k = torch.randn((600, 1, 64), generator=torch.Generator().manual_seed(1)).to(dev)
    slots = torch.arange(600).to(dev)

    def run(stream):
        cache = [torch.zeros((40, 1, 16, 64), dtype=torch.int8, device=dev) for _ in range(2)]
        scales = [torch.zeros((40, 1), device=dev) for _ in range(2)]
        if dev == "cuda":
            torch.cuda.synchronize()
        pa.pa_append_kv_block_quant(k, k, slots, *cache, *scales, stream=stream)
        if dev == "cuda":
            torch.cuda.synchronize()
        return cache[0]
    return run


@case
def decode(dev):
    g = torch.Generator().manual_seed(2)
    cache = torch.randint(-127, 128, (40, 2, 16, 64), generator=g).to(torch.int8).to(dev)
    scales = torch.rand((40, 2), generator=g).to(dev)
    q = torch.randn((2, 8, 64), generator=g).to(dev)
    tables = torch.arange(38, dtype=torch.int32).view(2, 19).contiguous().to(dev)
    lens = torch.tensor([300, 290], dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    return lambda stream: pa.pa_decode_block_quant(out, q, cache, cache, scales, scales, tables, lens, stream=stream)


def pages(dev):
    i32 = dict(dtype=torch.int32, device=dev)
    tables = torch.arange(12, **i32).view(3, 4).contiguous()
    return tables, torch.ones(20, **i32), torch.tensor([50, 64, 3], **i32), torch.empty(4, **i32)


@case
def update(dev):
    tables, refs, lens, status = pages(dev)
    refs[12:] = 0
    new, new_refs = torch.empty_like(tables), torch.empty_like(refs)
    pairs = torch.empty((3, 2), dtype=torch.int64, device=dev)
    return lambda stream: pa.pa_pages_update(new, new_refs, pairs, status, tables, refs, lens, lens - 1, lens, 16,
                                             stream=stream)


@case
def compact(dev):
    tables, refs, lens, status = pages(dev)
    new, new_refs, remap = torch.empty_like(tables), torch.empty_like(refs), torch.empty_like(refs)
    pairs = torch.empty((10, 2), dtype=torch.int64, device=dev)
    return lambda stream: pa.pa_pages_compact(new, new_refs, remap, pairs, status, tables, refs, lens, 16, stream=stream)


class Record:
    """Stands in for the library: every size query asks for 4096 bytes, every call succeeds."""

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 4096
        return lambda *a: pa.PA_OK


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_workspace_is_made_under_the_given_stream(name, monkeypatch):
    inside, made = [], []

    @contextlib.contextmanager
    def scope(stream):
        inside.append(stream)
        yield
        inside.pop()

    real = torch.empty

    def empty(*a, **kw):
        made.append(list(inside))
        return real(*a, **kw)

    stream = types.SimpleNamespace(cuda_stream=7, device_index=0, device=torch.device("cuda", 0))
    monkeypatch.setattr(torch.cuda, "stream", scope)
    monkeypatch.setattr(pa, "_lib", Record())
    monkeypatch.setattr(pa, "_dense", lambda *a: 0)
    monkeypatch.setattr(pa, "_call", lambda fn, dev, stream, *a: None)
    run = CALLS[name]("cpu")
    monkeypatch.setattr(torch, "empty", empty)
    run(stream)
    assert made == [[stream]]


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_side_stream_gives_the_same(name):
    run = CALLS[name]("cuda")
    torch.cuda.synchronize()
    want = run(None).clone()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(3):
        got = run(stream)
        after = [torch.empty(1 << 16, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del after
