"""Pins of oracle/options.py."""
import numpy as np
import pytest

from oracle.options import options_attention
from oracle.prefill import prefill_attention


def _qkv(n, L, hq, hkv, D=16, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((n, hq, D)), r.standard_normal((L, hkv, D)), r.standard_normal((L, hkv, D))


def test_everything_off_is_plain_causal_attention():
    q, K, V = _qkv(5, 9, 4, 2)
    out, lse, size = options_attention(q, K, V, 0.3)
    assert np.abs(out - prefill_attention(q, K, V, 0.3)).max() < 1e-14
    assert (size >= np.abs(out) - 1e-15).all()
    assert np.array_equal(options_attention(q, K, V, 0.3, window=9)[0], out)


@pytest.mark.parametrize("window,cap,sink", [(3, 0.0, None), (0, 2.0, None), (4, 1.5, -0.3), (1, 0.0, 2.0)])
def test_against_a_masked_matrix(window, cap, sink):
    q, K, V = _qkv(6, 11, 2, 1, seed=window)
    sinks = None if sink is None else np.array([sink, sink + 1])
    out, lse, _ = options_attention(q, K, V, 0.5, window, cap, sinks)
    p, j = np.arange(5, 11)[:, None], np.arange(11)[None]
    mask = (j <= p) & ((j > p - window) if window else True)
    for h in range(2):
        x = 0.5 * q[:, h] @ K[:, 0].T
        x = cap * np.tanh(x / cap) if cap else x
        e = np.where(mask, np.exp(x), 0.0)
        den = e.sum(1) + (0 if sinks is None else np.exp(sinks[h]))
        assert np.abs(out[:, h] - (e / den[:, None]) @ V[:, 0]).max() < 1e-13
        assert np.abs(lse[:, h] - np.log(den)).max() < 1e-13


def test_closed_forms():
    q, K, V = _qkv(3, 3, 1, 1)
    out, lse, _ = options_attention(q, K, V, 0.7, window=1)          # each sees itself alone
    assert np.abs(out[:, 0] - V[:, 0]).max() < 1e-15
    assert np.abs(lse[:, 0] - 0.7 * (q[:, 0] * K[:, 0]).sum(1)).max() < 1e-14
    half, _, _ = options_attention(q * 0, K, V, 1.0, window=1, sinks=[0.0])   # score 0 against a sink of 0
    assert np.abs(half[:, 0] - V[:, 0] / 2).max() < 1e-15
    gone, l2, _ = options_attention(q, K, V, 1.0, sinks=[1e4])
    assert np.abs(gone).max() == 0 and np.abs(l2 - 1e4).max() < 1e-9
    none, l3, _ = options_attention(q[:1], K[:0], V[:0], 1.0)
    assert not none.any() and l3[0, 0] == -np.inf
    _, l4, _ = options_attention(q[:2], K[:1], V[:1], 1.0, sinks=[0.25])      # the first token is before position 0
    assert l4[0, 0] == 0.25


@pytest.mark.parametrize("window,cap,sink", [(0, 0.0, None), (3, 0.0, 0.4), (7, 2.0, None), (1, 1.0, float("-inf"))])
def test_row_wise_and_matrix_forms_agree(window, cap, sink):
    from oracle.options import options_attention_masked
    q, K, V = _qkv(9, 13, 4, 2, seed=3)
    sinks = None if sink is None else np.full(4, sink)
    for a, b in zip(options_attention(q, K, V, 0.4, window, cap, sinks),
                    options_attention_masked(q, K, V, 0.4, window, cap, sinks)):
        assert np.abs(a - b).max() < 1e-13
