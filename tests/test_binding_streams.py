"""The binding's way to the current stream and device."""
import contextlib
import importlib.util
import types

import pytest
import torch

from paged_kv_cache_251_gb300 import pa

INNER = ("_cuda_getCurrentRawStream", "_cuda_getDevice")


def load(monkeypatch, drop):
    """The binding, loaded as on a torch without its inner names."""
    for name in INNER if drop else ():
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("pa_loaded_again", pa.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_a_torch_without_the_inner_names(monkeypatch):
    """The calls go by the public names then: same stream, same device switch."""
    m = load(monkeypatch, True)
    entered, got = [], []

    @contextlib.contextmanager
    def device(dev):
        entered.append(dev)
        yield

    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=100 + dev))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    m._call(lambda *a: got.append(a) or 0, 0, None, "x")
    assert got == [("x", 100)] and entered == []
    m._call(lambda *a: got.append(a) or 0, 1, None, "y")
    assert got[1] == ("y", 101) and entered == [1]


@pytest.mark.gpu
def test_both_ways_name_the_same(monkeypatch):
    x = torch.randn(5, 2, 64, device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    f = pa.pa_rope_frequencies(64).cuda()
    want = pa.pa_rope(torch.empty_like(x), x, pos, f)
    stream = torch.cuda.Stream()
    with monkeypatch.context() as patch:
        m = load(patch, True)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        assert m._raw_stream(0) == pa._raw_stream(0) == stream.cuda_stream
        out = m.pa_rope(torch.empty_like(x), x, pos, f)
    torch.cuda.synchronize()
    assert m._current_device() == pa._current_device() == 0 and torch.equal(out, want)
