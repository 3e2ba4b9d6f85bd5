"""pa_rotate_and_cache refuses bad arguments on the host, before any launch."""
import ctypes

import pytest
import torch

from paged_kv_cache_361_b200 import binding as B

OK = dict(q=16, qs=1024, k=16, ks=256, v=16, vs=256, pos=16, table=16, max_pos=8, rd=128, inter=0, slots=16, n=3, hq=8,
          qo=32)


def _call(cache_kw=None, **kw):
    a = dict(OK, **kw)
    c = B.pa_cache(**dict(dict(k=16, v=32, num_blocks=8, num_kv_heads=2, block_size=16, head_dim=128,
                               dtype=B.PA_BF16), **(cache_kw or {})))
    return B._lib().pa_rotate_and_cache(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["table"],
                                        a["max_pos"], a["rd"], a["inter"], a["slots"], a["n"], a["hq"],
                                        ctypes.byref(c), a["qo"], None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(max_pos=0), dict(inter=2), dict(hq=0), dict(hq=-1), dict(q=None), dict(qo=None), dict(k=None),
    dict(v=None), dict(pos=None), dict(table=None), dict(slots=None), dict(q=18), dict(k=24), dict(v=24), dict(qo=40),
    dict(table=24), dict(pos=18), dict(slots=12), dict(qs=1016), dict(qs=1028), dict(ks=248), dict(ks=260),
    dict(vs=128), dict(vs=257), dict(qo=16, qs=2048)])
def test_invalid_arguments(kw):
    assert _call(**kw) == B.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("rd", [0, 8, 24, 129, 144, 256, -16])
def test_rotary_dims_outside_the_set(rd):
    assert _call(rd=rd) == B.PA_ERR_UNSUPPORTED


def test_cache_checks_and_empty_call():
    assert _call(dict(head_dim=96)) == B.PA_ERR_UNSUPPORTED
    assert _call(dict(dtype=B.PA_INT8)) == B.PA_ERR_INVALID_ARG
    assert _call(hq=2 ** 27, qs=2 ** 34) == B.PA_ERR_UNSUPPORTED
    assert _call(n=0, k=None, v=None, pos=None, table=None, slots=None) == B.PA_OK


def test_token_rows_of_views():
    """(On the host, whose device index is -1.)"""
    dt = torch.bfloat16
    fused = torch.zeros(5, 12 * 64, dtype=dt)
    rows = lambda t, n=5: B._token_rows(t, "k", dt, n, 2, 64, -1)
    assert rows(fused[:, 128:256].unflatten(1, (2, 64))) == 768
    assert rows(fused[:, 128:256].unflatten(1, (2, 64))[:1], 1) == 128
    assert rows(torch.zeros(0, 2, 64, dtype=dt), 0) == 128
    for bad in (fused[:, :256:2].unflatten(1, (2, 64)), torch.zeros(5, 64, 2, dtype=dt).transpose(1, 2),
                torch.zeros(1, 2, 64, dtype=dt).expand(5, 2, 64), torch.zeros(5, 3, 64, dtype=dt),
                torch.zeros(4, 2, 64, dtype=dt), torch.zeros(5, 128, dtype=dt)):
        with pytest.raises(ValueError):
            rows(bad)
    for device_index, t in ((0, fused.unflatten(1, (12, 64))), (0, torch.zeros(5, 2, 64))):
        with pytest.raises(TypeError):
            B._token_rows(t, "k", dt, 5, 2, 64, device_index)
