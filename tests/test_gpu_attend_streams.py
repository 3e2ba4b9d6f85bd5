"""PagedKVCache.attend on several streams."""
import pytest
import torch

from paged_kv_cache_361_b200 import PagedKVCache

pytestmark = pytest.mark.gpu


def test_attend_on_two_streams_at_once():
    """One cache, one long sequence each, the calls queued behind one event: each
    stream's results are those of its calls alone."""
    g = torch.Generator().manual_seed(5)
    cache = PagedKVCache(3000, 2, 16, 64, torch.bfloat16, "cuda")
    for s in (0, 1):
        cache.add_sequence(s, *(torch.randn(20000, 2, 64, generator=g).bfloat16().cuda() for _ in "kv"))
    q = [torch.randn(1, 8, 64, generator=g).bfloat16().cuda() for _ in (0, 1)]
    want = [cache.attend([s], [1], q[s]) for s in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in (0, 1)]
    torch.cuda._sleep(20_000_000)                       # (some 10 ms, in which all calls below are queued)
    ready = torch.cuda.Event()
    ready.record()
    got = [[], []]
    for s in (0, 1):
        streams[s].wait_event(ready)
    for _ in range(20):
        for s in (0, 1):
            with torch.cuda.stream(streams[s]):
                got[s].append(cache.attend([s], [1], q[s]))
    torch.cuda.synchronize()
    for s in (0, 1):
        assert all(torch.equal(x, want[s]) for x in got[s])
