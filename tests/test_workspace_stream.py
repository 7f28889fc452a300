"""A workspace that a call makes for itself belongs to the stream the call runs on."""
import contextlib
import types

import pytest
import torch

import paged_kv_cache_251_gb300.pa as pa

CALLS = {}


def case(fn):
    CALLS[fn.__name__] = fn
    return fn


# Each case: the inputs on `dev`, two sequences of about 300 tokens, and a function
# that makes the call on a stream and returns its output.
def _paged(dev):
    cache = torch.randn(40, 2, 16, 128, generator=torch.Generator().manual_seed(1)).half()
    tables = torch.arange(38, dtype=torch.int32).view(2, 19).contiguous()
    return (cache.to(dev), cache.flip(0).contiguous().to(dev), tables.to(dev),
            torch.tensor([300, 290], dtype=torch.int32, device=dev))


def _normal(dev, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(2)).half().to(dev)


@case
def decode(dev):
    q, args = _normal(dev, 2, 8, 128), _paged(dev)
    out = torch.empty_like(q)
    return lambda stream: pa.pa_decode(out, q, *args, partition_size=64, stream=stream)


@case
def decode_shared_prefix(dev):
    q, (k, v, tables, lens) = _normal(dev, 2, 8, 128), _paged(dev)
    out, tables = torch.empty_like(q), torch.cat([tables[:1], tables[:1]]).contiguous()
    shared = torch.tensor([256], dtype=torch.int32, device=dev)
    return lambda stream: pa.pa_decode_shared_prefix(out, q, k, v, tables, lens, shared, 2, partition_size=64,
                                                     stream=stream)


@case
def decode_contiguous(dev):
    q, k, lens = _normal(dev, 2, 8, 128), _normal(dev, 2, 8, 304, 128), _paged(dev)[3]
    out = torch.empty_like(q)
    return lambda stream: pa.pa_decode_contiguous(out, q, k, k, lens, partition_size=64, stream=stream)


@case
def decode_quant(dev):
    q, (_, _, tables, lens) = _normal(dev, 2, 8, 128), _paged(dev)
    k = torch.ones(pa.quant_pool_shape(40, 2, 16, 128), dtype=torch.int8, device=dev)
    out = torch.empty_like(q)
    return lambda stream: pa.pa_decode_quant(out, q, k, k, tables, lens, partition_size=64, stream=stream)


@case
def decode_tree(dev):
    q, args = _normal(dev, 2, 3, 8, 128), _paged(dev)
    out = torch.empty_like(q)
    return lambda stream: pa.pa_decode_tree(out, q, *args, stream=stream)


@case
def decode_scored(dev):
    q, args, scores = _normal(dev, 2, 8, 128), _paged(dev), torch.zeros(2, 2, 304, device=dev)
    out = torch.empty_like(q)
    return lambda stream: pa.pa_decode_scored(out, scores, q, *args, partition_size=64, stream=stream)


class Record:
    """Stands in for the library: every size query asks for 4096 bytes, every call
    succeeds."""

    def __getattr__(self, name):
        real = getattr(LIB, name)
        if name.startswith("pa_decode") and name.endswith("workspace_size"):
            return lambda *a: 4096
        return (lambda *a: pa.PA_OK) if name.startswith("pa_decode") else real


LIB = pa._lib


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_workspace_is_made_under_the_given_stream(name, monkeypatch):
    """On the CPU, with the library, the device checks and the stream replaced."""
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
    monkeypatch.setattr(pa, "_cuda", lambda *a: None)
    monkeypatch.setattr(pa, "_dense", lambda *a: 0)
    monkeypatch.setattr(pa, "_call", lambda fn, dev, stream, *a: None)
    run = CALLS[name]("cpu")
    monkeypatch.setattr(torch, "empty", empty)
    run(stream)
    assert made == [[stream]]


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_workspace_comes_from_the_streams_own_memory(name, monkeypatch):
    """On the GPU: the block that the call asks for lies in memory the allocator keeps
    for the call's stream, so nothing on another stream is given it while the call
    runs; and the result is the default stream's, with such allocations made and
    written right after the call."""
    run = CALLS[name]("cuda")
    want = run(None).clone()
    stream = torch.cuda.Stream()
    real, made = torch.empty, []

    def empty(*a, **kw):
        t = real(*a, **kw)
        made.append((t.data_ptr(), t.numel() * t.element_size()))
        return t

    torch.cuda.synchronize()
    for _ in range(5):
        made.clear()
        with monkeypatch.context() as m:
            m.setattr(torch, "empty", empty)
            got = run(stream)
        assert len(made) == 1
        at, size = made[0]
        after = [real(size, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(4)]
        homes = [s["stream"] for s in torch.cuda.memory_snapshot()
                 if s["address"] <= at < s["address"] + s["total_size"]]
        assert homes == [stream.cuda_stream]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del after
