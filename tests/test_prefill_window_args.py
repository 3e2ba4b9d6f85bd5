"""pa_prefill_window refuses bad arguments on the host, before any launch."""
import ctypes

import pytest

from paged_kv_cache_361_b200 import binding as B

OK = dict(q=16, T=600, n=3, cu=16, mq=400, hq=8, tables=16, mb=64, lens=16, mc=1000, scale=0.1, out=16, window=0,
          cap=0.0, sinks=None, lse=None)


def _call(cache_kw=None, no_options=False, **kw):
    a = dict(OK, **kw)
    c = B.pa_cache(**dict(dict(k=16, v=32, num_blocks=8, num_kv_heads=2, block_size=16, head_dim=128,
                               dtype=B.PA_BF16), **(cache_kw or {})))
    o = B.pa_attn_options(a["window"], a["cap"], a["sinks"], a["lse"])
    return B._lib().pa_prefill_window(a["q"], a["T"], a["n"], a["cu"], a["mq"], a["hq"], ctypes.byref(c), a["tables"],
                                      a["mb"], a["lens"], a["mc"], a["scale"],
                                      None if no_options else ctypes.byref(o), a["out"], None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(n=-1), dict(mq=-1), dict(mq=1001), dict(hq=0), dict(hq=9), dict(mb=0), dict(mc=-1), dict(mc=1025),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
    dict(cap=-1.0), dict(cap=float("inf")), dict(cap=float("nan")),
    dict(cap=2.0 ** 41), dict(cap=2.0 ** -41), dict(sinks=18), dict(lse=18), dict(q=None),
    dict(q=24), dict(cu=18), dict(cu=None), dict(tables=None), dict(tables=18), dict(lens=None), dict(lens=18),
    dict(out=None), dict(out=24)])
def test_invalid_arguments(kw):
    assert _call(**kw) == B.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,cache", [
    (dict(hq=6), {}), (dict(hq=32), {}), ({}, dict(block_size=4)), ({}, dict(dtype=B.PA_F32)), ({}, dict(head_dim=256)),
    ({}, dict(num_blocks=2 ** 28)), (dict(n=65536), {}), (dict(mc=2 ** 30 + 1, mb=2 ** 27), {}),
    (dict(mq=2 ** 24, mc=2 ** 24, mb=2 ** 20), {})])
def test_unsupported(kw, cache):
    assert _call(cache, **kw) == B.PA_ERR_UNSUPPORTED


def test_empty_calls():
    for kw in (dict(n=0), dict(T=0), dict(mq=0)):
        assert _call(no_options=True, q=None, out=None, **kw) == B.PA_OK
