"""Pins of oracle/rotary.py and of rotary_table, on the CPU."""
import numpy as np
import pytest

from oracle.rotary import rotate
from paged_kv_cache_361_b200 import binding as B


def _angles(pos, rd, base=10000.0):
    return np.outer(pos, base ** (-np.arange(0, rd, 2) / rd))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rd", [16, 48, 64])
def test_rotation_is_complex_multiplication(rd, interleaved):
    rng = np.random.default_rng(rd)
    x = rng.standard_normal((5, 3, 64))
    th = _angles(rng.integers(0, 100000, 5), rd)
    y = rotate(x, np.cos(th), np.sin(th), interleaved)
    a, b = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * th)[:, None]
    assert np.abs(y[..., a] - z.real).max() < 1e-14 and np.abs(y[..., b] - z.imag).max() < 1e-14
    assert np.array_equal(y[..., rd:], x[..., rd:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_dot_products_depend_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))

    def dot(pq, pk):
        tq, tk = _angles([pq], 64), _angles([pk], 64)
        return float((rotate(q, np.cos(tq), np.sin(tq), interleaved) *
                      rotate(k, np.cos(tk), np.sin(tk), interleaved)).sum())
    assert abs(dot(5, 3) - dot(1005, 1003)) < 1e-10
    assert abs(dot(0, 0) - float((q * k).sum())) < 1e-14


def test_rotary_table_is_exact_at_far_positions():
    """Every entry is the fp32 nearest the 64-bit value: half a step, with the
    angle's own 64-bit rounding (2^-53 * 3e5) far below it."""
    t = B.rotary_table(300000, 64, 10000.0, device="cpu").numpy().astype(np.float64)
    pos = np.array([0, 1, 77, 131071, 299999])
    th = _angles(pos, 64)
    ref = np.concatenate([np.cos(th), np.sin(th)], 1)
    assert np.abs(t[pos] - ref).max() <= 2.0 ** -25 + 1e-10
    assert t.shape == (300000, 64)
