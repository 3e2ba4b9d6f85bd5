"""Oracle for attention with a sliding window, capped scores, sinks and the
log-sum-exp. TEST INFRASTRUCTURE ONLY.

The new token at position p (the last n of L) sees the keys p - window < j <= p
(window 0: j <= p), of score x = scale q.k, or cap tanh(scale q.k / cap):
  den = sum_j exp(x_j) + exp(sink);  out = sum_j exp(x_j) v_j / den;  lse = log den.
A token that sees no key gives zeros, and lse = sink (or -inf).
"""
from __future__ import annotations

import numpy as np

from .attention import _f64


def options_attention(q, K, V, scale: float, window: int = 0, cap: float = 0.0, sinks=None):
    """q [n][Hq][D]; K, V [L][Hkv][D] in logical order. Returns (out, lse, size):
    out [n][Hq][D], lse [n][Hq] and size = the same average of |V|, which the
    rounding of weights is measured by."""
    q, K, V = _f64(q), _f64(K), _f64(V)
    n, hq, d = q.shape
    L, hkv = K.shape[0], K.shape[1]
    out, size, lse = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    for i in range(n):
        p = L - n + i
        lo = max(0, p - window + 1) if window else 0
        for h in range(hq):
            x = np.empty(0)
            if p >= 0:
                kk, vv = K[lo:p + 1, h // (hq // hkv)], V[lo:p + 1, h // (hq // hkv)]
                x = scale * (kk @ q[i, h])
                if cap:
                    x = cap * np.tanh(x / cap)
            sink = -np.inf if sinks is None else float(sinks[h])
            top = max(x.max(initial=-np.inf), sink)
            if top == -np.inf:
                continue
            den = np.exp(x - top).sum() + np.exp(sink - top)
            lse[i, h] = top + np.log(den)
            if len(x):
                w = np.exp(x - top) / den
                out[i, h], size[i, h] = w @ vv, w @ np.abs(vv)
    return out, lse, size


def options_attention_masked(q, K, V, scale: float, window: int = 0, cap: float = 0.0, sinks=None):
    """The same written as one masked matrix softmax per head, for long prompts
    (an independent form, used to pin the row-wise one too)."""
    q, K, V = _f64(q), _f64(K), _f64(V)
    n, hq, d = q.shape
    L, hkv = K.shape[0], K.shape[1]
    p, j = np.arange(L - n, L)[:, None], np.arange(L)[None]
    seen = (j <= p) & (j > p - window) if window else j <= p
    out, size, lse = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.empty((n, hq))
    for h in range(hq):
        x = scale * q[:, h] @ K[:, h // (hq // hkv)].T
        x = np.where(seen, cap * np.tanh(x / cap) if cap else x, -np.inf)
        if sinks is not None:
            x = np.concatenate([x, np.full((n, 1), float(sinks[h]))], 1)
        top = x.max(1, keepdims=True, initial=-1e300)
        e = np.exp(x - top)
        den = e.sum(1, keepdims=True)
        with np.errstate(divide="ignore"):
            lse[:, h] = (np.where(den > 0, top, -np.inf) + np.log(np.where(den > 0, den, 1.0)))[:, 0]
        w = e[:, :L] / np.where(den > 0, den, 1.0)
        v = V[:, h // (hq // hkv)]
        out[:, h], size[:, h] = w @ v, w @ np.abs(v)
    return out, lse, size
