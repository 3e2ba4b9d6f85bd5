"""What PagedKVCache.attend asks of the native calls, on the host, with the device
calls replaced."""
import contextlib
import types

import pytest
import torch

from paged_kv_cache_361_b200 import PagedKVCache, binding as B, cache as cache_module

SIZES = (4, 4, 1, 32, 8, 64, 4096)


@pytest.fixture
def host_cache(monkeypatch):
    """A cache in host memory with a sequence of 100 tokens."""
    real = torch.empty
    monkeypatch.setattr(cache_module.torch, "empty", lambda *a, pin_memory=False, **kw: real(*a, **kw))
    cache = PagedKVCache(8, 2, 16, 64, torch.bfloat16, "cpu")
    cache.reserve(0, 100)
    return cache


def _two_devices(monkeypatch):
    """Device 0, the current one, whose plans need 100 bytes, and device 1 (900 bytes)."""
    now = [0]

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], torch.device(d).index
        yield
        now[0] = before
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(B, "_lib", lambda: types.SimpleNamespace(
        pa_decode_multi_workspace_bytes=lambda *a: (100, 900)[now[0]]))
    return now


def test_workspace_bytes_of_a_device(monkeypatch):
    now = _two_devices(monkeypatch)
    f = B.pa_decode_multi_workspace_bytes
    for device, want in ((None, 100), (torch.device("cuda:0"), 100), (torch.device("cuda:1"), 900),
                         (torch.device("cuda"), 100), ("cuda:1", 900)):
        assert f(*SIZES, device=device) == want and now == [0]
    assert f(*SIZES) == 100


def test_attend_plans_for_its_cache_s_device(monkeypatch, host_cache):
    """The plan depends on the number of SMs, and pa_decode_multi makes it on the cache's device."""
    tables = host_cache.decode_inputs([0])
    monkeypatch.setattr(host_cache, "decode_inputs", lambda ids: tables)
    _two_devices(monkeypatch)
    asked = []
    monkeypatch.setattr(host_cache, "workspace", asked.append)
    monkeypatch.setattr(B, "pa_decode_multi", lambda *a, **kw: None)
    host_cache.k_cache = types.SimpleNamespace(shape=host_cache.k_cache.shape, device=torch.device("cuda:1"))
    host_cache.attend([0], [1], torch.zeros(1, 4, 64, dtype=torch.bfloat16))
    assert asked == [900]


def test_streams_do_not_share_a_workspace(monkeypatch, host_cache):
    """Calls that share one must not overlap on the GPU; those of two streams may."""
    now = [11]
    monkeypatch.setattr(B, "_stream_on", lambda *a: now[0])
    first = host_cache.workspace(1000)
    assert host_cache.workspace(600) is first and host_cache.workspace(0) is None
    now[0] = 22
    other = host_cache.workspace(1000)
    assert other.data_ptr() != first.data_ptr()
    larger = host_cache.workspace(5000)
    assert larger.numel() >= 5000
    now[0] = 11
    assert host_cache.workspace(1000) is first
    now[0] = 22
    assert host_cache.workspace(1000) is larger
