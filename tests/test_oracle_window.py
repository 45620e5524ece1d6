"""Pins of the windowed oracle: the mask by definition, full attention where
the window covers everything, gradients against differences."""

import numpy as np
import pytest

import oracle
from oracle.window import allowed

rng = np.random.default_rng(0)


def _inputs(B, S, H, Hk, D):
    return [rng.standard_normal((B, S, h, D)) for h in (H, Hk, Hk, H)]


def test_mask_by_definition():
    for w in (1, 3, 100):
        for k in (0, 2, 50):
            got = allowed(np.arange(8), np.arange(8), w, k)
            for i in range(8):
                for j in range(8):
                    assert got[i, j] == (j <= i and (i - j < w or j < k))


@pytest.mark.parametrize("window,n_sink", [(20, 0), (99, 3), (1, 20)])
def test_all_tokens_visible_is_full_attention(window, n_sink):
    q, k, v, do = _inputs(2, 20, 4, 2, 16)
    out, lse = oracle.window_attention(q, k, v, window, n_sink, 0.25)
    want, want_l = oracle.attention_naive(q, k, v, True, 0.25)
    np.testing.assert_allclose(out, want, atol=1e-12)
    np.testing.assert_allclose(lse, want_l, atol=1e-12)
    for a, b in zip(oracle.window_backward(q, k, v, do, window, n_sink, 0.25),
                    oracle.attention_backward(q, k, v, do, True, 0.25)):
        np.testing.assert_allclose(a, b, atol=1e-12)


def test_window_of_one_is_the_token_itself():
    q, k, v, _ = _inputs(1, 6, 2, 2, 8)
    out, _ = oracle.window_attention(q, k, v, 1, 0, 1.0)
    np.testing.assert_allclose(out, v, atol=1e-12)


@pytest.mark.parametrize("window,n_sink", [(3, 2), (4, 0)])
def test_gradients_against_differences(window, n_sink):
    q, k, v, do = _inputs(1, 9, 2, 1, 4)
    grads = oracle.window_backward(q, k, v, do, window, n_sink, 0.5)
    loss = lambda: (oracle.window_attention(q, k, v, window, n_sink, 0.5)[0] * do).sum()   # noqa: E731
    for x, g in zip((q, k, v), grads):
        for idx in [(0, 0, 0, 1), (0, 4, 0, 0), (0, 8, 0, 3), (0, 1, 0, 2)]:
            keep, eps = x[idx], 1e-6
            x[idx] = keep + eps
            up = loss()
            x[idx] = keep - eps
            down = loss()
            x[idx] = keep
            assert abs((up - down) / (2 * eps) - g[idx]) < 1e-7


def test_packed_sequences_are_their_own():
    lengths = [5, 0, 1, 7]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    q, k, v, do = [rng.standard_normal((13, h, 8)) for h in (4, 2, 2, 4)]
    out, lse = oracle.window_attention_varlen(q, k, v, cu, 3, 1, 0.3)
    grads = oracle.window_backward_varlen(q, k, v, do, cu, 3, 1, 0.3)
    assert out.shape == q.shape and lse.shape == (4, 13)
    o, _ = oracle.window_attention(q[None, 6:], k[None, 6:], v[None, 6:], 3, 1, 0.3)
    np.testing.assert_array_equal(out[6:], o[0])
    g = oracle.window_backward(q[None, 6:], k[None, 6:], v[None, 6:], do[None, 6:], 3, 1, 0.3)
    for a, b in zip(grads, g):
        np.testing.assert_array_equal(a[6:], b[0])
