"""Oracle for rotary positions. TEST INFRASTRUCTURE ONLY.

Pair i of a head at position p is turned by the angle p * base^(-2i / rotary_dim):
(a', b') = (a cos - b sin, b cos + a sin). The pairs are dims (i, i + rotary_dim / 2)
or, interleaved, dims (2i, 2i + 1); the dims from rotary_dim on stay.

`rotate` computes in the dtype it is given: fp64 for values, fp32 for the bits
of an operator that rounds every product and sum to fp32.
"""
from __future__ import annotations

import numpy as np


def pair_dims(rotary_dim: int, interleaved: bool):
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def rotate(x, cos, sin, interleaved: bool) -> np.ndarray:
    """x [T][H][D], cos and sin [T][rotary_dim / 2], all of one dtype."""
    a_dims, b_dims = pair_dims(2 * cos.shape[1], interleaved)
    y = x.copy()
    c, s = cos[:, None], sin[:, None]
    a, b = x[..., a_dims], x[..., b_dims]
    y[..., a_dims] = a * c - b * s
    y[..., b_dims] = b * c + a * s
    return y
