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
