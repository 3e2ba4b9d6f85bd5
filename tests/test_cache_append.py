"""PagedKVCache.append_rotated is all or nothing: whatever fails, the block manager and
the lengths are as before. On CPU tensors, the device calls replaced."""
import numpy as np
import pytest
import torch

from paged_kv_cache_361_b200 import PagedKVCache, binding as B, cache as cache_module


class _Boom(RuntimeError):
    pass


@pytest.fixture
def layer(monkeypatch):
    """A cache of 6 blocks of 16 with sequence 0 (30 tokens) and its fork 1, what the
    replaced calls were given, and a switch that lets the n-th allocation from now on
    fail, of host or device memory alike."""
    calls, left, keep, real_on = [], [None], [], B._on

    def allocate(real):
        def f(*a, **kw):
            if left[0] is not None:
                left[0] -= 1
                if left[0] < 0:
                    raise _Boom
            kw.pop("pin_memory", None)
            return real(*a, **kw)
        return f
    monkeypatch.setattr(B, "_call_on", lambda *a: calls.append(("rotate", a)))
    monkeypatch.setattr(B, "_on", lambda t, *a: keep.append(t) or real_on(t, *a))
    monkeypatch.setattr(B, "_stream_on", lambda *a: 0)
    monkeypatch.setattr(B, "pa_copy_blocks", lambda *a: calls.append(("copy", a)))
    monkeypatch.setattr(B, "make_cache", lambda k, v: _struct(k, {}))
    monkeypatch.setattr(cache_module.torch, "empty", allocate(torch.empty))
    cache = PagedKVCache(6, 2, 16, 64, torch.bfloat16, "cpu")
    cache.reserve(0, 30)
    cache.fork(0, 1)

    def fail_after(n):
        left[0] = n
    return cache, calls, fail_after, keep


TABLE = torch.zeros(200, 64)


def _rows(n, heads=2):
    return torch.zeros(n, heads, 64, dtype=torch.bfloat16)


def _state(cache):
    return dict(cache.lens), cache.bm.stats(), [cache.bm.block_table(s)[0].tolist() for s in sorted(cache.lens)]


def test_an_allocation_that_fails_changes_nothing(layer):
    cache, calls, fail_after, keep = layer
    before = _state(cache)
    for n in range(50):
        fail_after(n)
        try:
            cache.append_rotated([0, 7], [3, 5], _rows(8, 4), _rows(8), _rows(8), TABLE)
        except _Boom:
            assert _state(cache) == before and not calls
            continue
        break
    else:
        raise AssertionError("never ran through")
    assert n >= 3                                  # q_out, and both sides of the upload
    fail_after(None)
    assert cache.lens == {0: 33, 1: 30, 7: 5}
    assert [c[0] for c in calls] == ["copy", "rotate"]
    pairs, (pos, slots) = calls[0][1][2], keep[-2:]
    assert pairs.shape == (1, 2) and pos.tolist() == [30, 31, 32, 0, 1, 2, 3, 4]
    block = lambda s, i: int(cache.bm.block_table(s)[0][i])
    assert slots.tolist() == [16 * block(0, 1) + 14, 16 * block(0, 1) + 15, 16 * block(0, 2)] + \
        [16 * block(7, 0) + i for i in range(5)]
    assert pairs.tolist() == [[block(1, 1), block(0, 1)]]


@pytest.mark.parametrize("ids", [[7, "8"], [7, np.int64(8), None], [7, 8.5]])
def test_an_identifier_that_is_none_changes_nothing(layer, ids):
    """A sequence that was made for a call that fails is given back whatever it fails with."""
    cache, calls, *_ = layer
    before = _state(cache)
    T = 2 * len(ids)
    with pytest.raises(Exception):
        cache.append_rotated(ids, [2] * len(ids), _rows(T, 4), _rows(T), _rows(T), TABLE)
    assert _state(cache) == before and not calls


def test_no_blocks_left_changes_nothing(layer):
    cache, calls, *_ = layer
    before = _state(cache)
    with pytest.raises(B.PagedAttnError):
        cache.append_rotated([7, 0], [16, 90], _rows(106, 4), _rows(106), _rows(106), TABLE)
    assert _state(cache) == before and not calls


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), B.PA_ERR_UNSUPPORTED), (dict(block_size=24), B.PA_ERR_UNSUPPORTED),
    (dict(dtype=torch.int8, k_scale=0.0), B.PA_ERR_INVALID_ARG),
    (dict(dtype=torch.float8_e4m3fn, v_scale=float("nan")), B.PA_ERR_INVALID_ARG)])
def test_a_cache_that_the_native_call_refuses_changes_nothing(monkeypatch, layer, kw, status):
    args = dict(dict(num_blocks=6, num_kv_heads=2, block_size=16, head_dim=64, dtype=torch.bfloat16, device="cpu"), **kw)
    cache = PagedKVCache(**args)
    monkeypatch.setattr(B, "make_cache", lambda k, v: _struct(k, kw))
    d = args["head_dim"]
    rows = lambda h: torch.zeros(5, h, d, dtype=torch.bfloat16)
    with pytest.raises(B.PagedAttnError) as e:
        cache.append_rotated([0], [5], rows(4), rows(2), rows(2), torch.zeros(20, 64))
    assert e.value.status == status
    assert cache.lens == {} and cache.bm.stats()["free_blocks"] == 6


def _struct(k_cache, kw):
    dtype = {torch.bfloat16: B.PA_BF16, torch.int8: B.PA_INT8, torch.float8_e4m3fn: B.PA_FP8_E4M3}[k_cache.dtype]
    return B.pa_cache(16, 32, *k_cache.shape, dtype, kw.get("k_scale", 1.0), kw.get("v_scale", 1.0))
