"""Numbers that pa_decode_multi, pa_prefill_window and their bindings refuse, on the
host before any launch."""
import ctypes

import pytest

from paged_kv_cache_361_b200 import binding as B


def _calls(scale, cap, dtype=B.PA_BF16, k_scale=1.0):
    """Status of both entry points for a call without sequences' rows to work on, so
    that what is not refused returns before any launch."""
    c = B.pa_cache(16, 32, 8, 2, 16, 128, dtype, k_scale, 1.0)
    o = ctypes.byref(B.pa_attn_options(0, cap, None, None))
    return (B._lib().pa_decode_multi(16, 0, 3, 16, 4, 8, ctypes.byref(c), 16, 64, 16, 1000, scale, o, 16, -1, 256,
                                     1 << 30, None),
            B._lib().pa_prefill_window(16, 0, 3, 16, 400, 8, ctypes.byref(c), 16, 64, 16, 1000, scale, o, 16, None))


@pytest.mark.parametrize("scale,cap,k_scale", [
    (1e-39, 0.0, 1.0),              # scale log2 e is below 2^-126
    (3e38, 0.0, 1.0),               # and above fp32's range
    (0.088, 0.0, 1e-38), (0.088, 0.0, 1e-45), (0.088, 0.0, 3e38 / 0.088), (1e20, 0.0, 1e20),
    (0.088, 2.0 ** 40, 3e-33),      # scale / cap k_scale is 0
    (1e-30, 2.0 ** 40, 1.0), (1e30, 2.0 ** -40, 1.0), (0.088, 2.0 ** -40, 1e30),
    (1.5e38 * 2.0 ** -40, 2.0 ** -40, 1.0)])  # scale / cap is in range, its product with 2 log2 e is not
def test_products_of_the_scales_outside_normal_fp32_are_refused(scale, cap, k_scale):
    """(A masked score, -inf, times a product that has become 0 is NaN.)"""
    assert _calls(scale, cap, B.PA_FP8_E4M3, k_scale) == (B.PA_ERR_INVALID_ARG,) * 2
    assert _calls(scale, cap, B.PA_INT8, k_scale) == (B.PA_ERR_INVALID_ARG,) * 2
    if k_scale == 1.0:
        assert _calls(scale, cap) == (B.PA_ERR_INVALID_ARG,) * 2


@pytest.mark.parametrize("scale,cap,k_scale", [
    (0.088, 0.0, 1.0), (1e-37, 0.0, 1.0), (1e38, 0.0, 1.0), (0.088, 2.0 ** 40, 1e-24), (0.088, 2.0 ** -40, 1e24),
    (0.088, 0.0, 3e-33), (2e-38, 2.0 ** -40, 1.0)])   # (with a cap, scale log2 e is not used)
def test_products_inside_it_are_taken(scale, cap, k_scale):
    assert _calls(scale, cap, B.PA_FP8_E4M3, k_scale) == (B.PA_OK,) * 2
    if k_scale == 1.0:
        assert _calls(scale, cap) == (B.PA_OK,) * 2


def test_k_scale_of_a_bf16_cache_is_not_looked_at():
    assert _calls(0.088, 0.0, B.PA_BF16, 1e-45) == (B.PA_OK,) * 2




@pytest.fixture
def host_calls(monkeypatch):
    """The bindings on CPU tensors (device index -1) up to the native call, whose
    arguments are returned as that call gets them."""
    import torch
    seen = {}

    def record(device_index, fn, what, *args):
        seen[what] = [a if isinstance(a, (int, float)) and not isinstance(a, bool) else None for a in args]
        for a, t in zip(args, B._SIGS[what][1]):
            if t in (ctypes.c_int32, ctypes.c_int64, ctypes.c_float):
                t.from_param(a)                    # ctypes takes it
    monkeypatch.setattr(B, "_call_on", record)
    monkeypatch.setattr(B, "_stream_on", lambda *a: 0)
    monkeypatch.setattr(B, "make_cache", lambda k, v: B.pa_cache(16, 32, *k.shape, B.PA_BF16, 1.0, 1.0))
    kc, vc = (torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16) for _ in "kv")
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    args = dict(q=q, cu_q_lens=i32(0, 2, 4), k_cache=kc, v_cache=vc, block_tables=torch.zeros(2, 4, dtype=torch.int32),
                context_lens=i32(50, 60), scale=0.125, out=torch.zeros_like(q), max_q_len=2, max_context_len=64)

    def call(name, **kw):
        getattr(B, name)(**dict(args, **kw))
        return seen[name]
    return call


BOTH = ["pa_decode_multi", "pa_prefill_window"]


@pytest.mark.parametrize("name", BOTH)
@pytest.mark.parametrize("key", ["window", "max_q_len", "max_context_len"])
@pytest.mark.parametrize("value", [2 ** 32 + 7, 2 ** 32, 2 ** 31, -2 ** 31 - 1, 10 ** 30])
def test_whole_numbers_outside_32_bits_are_refused(host_calls, name, key, value):
    """(ctypes keeps the low 32 bits: a window of 2^32 + 7 would be one of 7.)"""
    with pytest.raises(ValueError, match=key):
        host_calls(name, **{key: value})


def test_partition_tokens_and_workspace_sizes_outside_32_bits(host_calls):
    with pytest.raises(ValueError, match="partition_tokens"):
        host_calls("pa_decode_multi", partition_tokens=2 ** 32 + 64)
    good = (4, 4, 1, 32, 8, 64, 4096, 1000, 512)
    assert B.pa_decode_multi_workspace_bytes(*good) > 0
    for i in range(len(good)):
        with pytest.raises(ValueError):
            B.pa_decode_multi_workspace_bytes(*[2 ** 32 + x if j == i else x for j, x in enumerate(good)])


@pytest.mark.parametrize("name", BOTH)
def test_numpy_and_torch_numbers_are_taken(host_calls, name):
    """As the other calls take them."""
    import numpy as np
    import torch
    want = host_calls(name, window=33)
    for whole, real in ((np.int64, np.float32), (np.int32, np.float64), (torch.tensor, torch.tensor)):
        got = host_calls(name, window=whole(33), max_q_len=whole(2), max_context_len=whole(64), scale=real(0.125),
                         softcap=real(0.0))
        assert got == want
    assert B.pa_decode_multi_workspace_bytes(*[np.int64(x) for x in (4, 4, 1, 32, 8, 64, 4096, 0, -1)]) == \
        B.pa_decode_multi_workspace_bytes(4, 4, 1, 32, 8, 64, 4096, 0, -1)
    for bad in (2.0, "2", None):
        with pytest.raises(TypeError):
            host_calls(name, max_q_len=bad)


@pytest.mark.parametrize("name", BOTH)
@pytest.mark.parametrize("cap", [1e-46, -1e-46, 2.0 ** -41, 1e39, float("nan"), float("inf"), -1.0])
def test_caps_are_checked_before_they_are_rounded(host_calls, name, cap):
    """(1e-46 is 0 in fp32, which means no cap.)"""
    with pytest.raises(B.PagedAttnError) as e:
        host_calls(name, softcap=cap)
    assert e.value.status == B.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", BOTH)
@pytest.mark.parametrize("key", ["q", "out", "block_tables", "context_lens", "sinks", "lse"])
def test_what_is_no_tensor_is_a_type_error(host_calls, name, key):
    import numpy as np
    for value in ([1, 2], np.zeros(4, dtype=np.float32)) + (() if key in ("sinks", "lse") else (None,)):
        with pytest.raises(TypeError, match=key):
            host_calls(name, **{key: value})


@pytest.mark.parametrize("key", ["q", "k", "v", "q_out", "positions", "slot_mapping", "cos_sin"])
def test_what_is_no_tensor_is_a_type_error_of_the_rotation(host_calls, key):
    import numpy as np
    import torch
    rows = lambda h: torch.zeros(3, h, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    args = dict(q=rows(4), k=rows(2), v=rows(2), positions=torch.zeros(3, dtype=torch.int32), cos_sin=torch.zeros(9, 64),
                slot_mapping=torch.zeros(3, dtype=torch.int64), k_cache=cache, v_cache=cache.clone(), q_out=rows(4))
    B.pa_rotate_and_cache(**args)
    for value in ([1, 2], np.zeros((3, 2, 64), dtype=np.float32)) + (() if key in ("q", "q_out") else (None,)):
        with pytest.raises(TypeError, match=key):
            B.pa_rotate_and_cache(**dict(args, **{key: value}))
