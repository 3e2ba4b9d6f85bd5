"""pa_decode_multi and pa_decode_multi_workspace_bytes on the host: refusals
before any launch, and what a split needs."""
import ctypes

import pytest

from paged_kv_cache_361_b200 import binding as B

OK = dict(q=16, T=6, n=3, cu=16, mq=4, hq=8, tables=16, mb=64, lens=16, mc=1000, scale=0.1, out=16, P=-1, ws=256,
          wsb=1 << 30, window=0, cap=0.0, sinks=None, lse=None)


def _call(cache_kw=None, no_options=False, **kw):
    a = dict(OK, **kw)
    c = B.pa_cache(**dict(dict(k=16, v=32, num_blocks=8, num_kv_heads=2, block_size=16, head_dim=128,
                               dtype=B.PA_BF16), **(cache_kw or {})))
    o = B.pa_attn_options(a["window"], a["cap"], a["sinks"], a["lse"])
    return B._lib().pa_decode_multi(a["q"], a["T"], a["n"], a["cu"], a["mq"], a["hq"], ctypes.byref(c), a["tables"],
                                    a["mb"], a["lens"], a["mc"], a["scale"], None if no_options else ctypes.byref(o),
                                    a["out"], a["P"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(n=-1), dict(mq=0), dict(mq=-3), dict(hq=0), dict(hq=9), dict(mb=0), dict(mc=-1), dict(mc=1025),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(P=-2), dict(P=32),
    dict(P=100), dict(window=-1), dict(cap=-1.0), dict(cap=float("inf")), dict(cap=float("nan")),
    dict(cap=2.0 ** 41), dict(cap=2.0 ** -41), dict(sinks=18),
    dict(lse=18), dict(q=None), dict(q=24), dict(cu=18), dict(tables=None), dict(tables=18), dict(lens=None),
    dict(lens=18), dict(out=None), dict(out=24), dict(ws=None), dict(ws=128), dict(wsb=64), dict(cu=None),
    dict(cu=None, mq=1, T=2)])
def test_invalid_arguments(kw):
    assert _call(**kw) == B.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,cache", [
    (dict(mq=17), {}), (dict(hq=6), {}), (dict(hq=32), {}), ({}, dict(block_size=4)), ({}, dict(dtype=B.PA_F32)),
    ({}, dict(head_dim=256)), ({}, dict(num_blocks=2 ** 28)), (dict(mc=2 ** 30 + 1, mb=2 ** 27), {}),
    (dict(n=2 ** 30, T=2 ** 30, P=0), {})])
def test_unsupported(kw, cache):
    assert _call(cache, **kw) == B.PA_ERR_UNSUPPORTED


def test_empty_calls():
    assert _call(n=0, q=None, out=None) == B.PA_OK
    assert _call(T=0, q=None, out=None, no_options=True) == B.PA_OK


def test_workspace_bytes():
    """Two partials a worker, (m, l) and o, of the rows of a (sequence, kv head)."""
    f = B.pa_decode_multi_workspace_bytes
    need = lambda workers, rows, D: -(-2 * workers * rows * 8 // 256) * 256 + 2 * workers * rows * D * 4
    assert f(4, 4, 1, 32, 8, 128, 4096, 0, 0) == 0                        # not split
    assert f(4, 4, 1, 32, 8, 128, 1, 0) == 0                              # one chunk a sequence
    assert f(4, 4, 1, 32, 8, 128, 4096, 0) == need(444, 4, 128)           # 3 CTAs per SM
    assert f(20, 4, 5, 32, 8, 128, 4096, 0) == need(148, 20, 128)         # on tcgen05: one
    assert f(4, 4, 1, 32, 8, 64, 257, 0) == need(4 * 8 * 5, 4, 64)        # fewer chunks of 64 than workers
    assert f(4, 4, 1, 32, 8, 64, 256, 0) == 0                             # no unit longer than the least share
    assert f(4, 4, 1, 32, 8, 64, 0, 0) == 0
    assert f(60, 60, 1, 64, 8, 64, 256, 0) == need(444, 8, 64)            # but more units than CTAs
    assert f(4, 4, 1, 32, 8, 128, 4096, 1000, 512) == need(4 * 8 * 9 // 4, 4, 128)   # 1000 + 63 keys in 128s, 4 a share
    for bad in ((0, 4, 1, 32, 8, 128, 4096), (4, 4, 17, 32, 8, 128, 4096), (4, 4, 1, 30, 8, 128, 4096),
                (4, 4, 1, 32, 8, 128, -1), (4, 4, 1, 32, 8, 128, 2 ** 30 + 1)):
        assert f(*bad) == 0
