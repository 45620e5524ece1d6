"""Pins of the 4-bit cache's oracle (oracle/kv4.py): rounding and format
against hand values and torch's conversions, attention against the full
attention oracle, eviction against brute force."""

import itertools

import numpy as np
import pytest
import torch

import oracle
from oracle import kv4


def test_bf16_rounding_equals_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4096), [0.0, -0.0, 1.00390625, 1.01171875, 3e38, 1e-40]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    np.testing.assert_array_equal(kv4.bf16(x), want)


def test_hand_quantised_group():
    # -8 .. 7 in steps of one: scale 1, zero 0, every value exact
    x = np.tile(np.arange(-8, 8), 4).astype(np.float32)
    codes, scale, zero = kv4.quantise(x)
    assert scale.tolist() == [1.0] and zero.tolist() == [0.0]
    np.testing.assert_array_equal(codes, np.tile(np.arange(16), 4))
    np.testing.assert_array_equal(kv4.values(codes, scale, zero), x)
    # a constant group: scale 0, code 8, the value itself (bf16)
    codes, scale, zero = kv4.quantise(np.full(64, 2.5, np.float32))
    assert scale[0] == 0 and zero[0] == 2.5 and (codes == 8).all()
    # not finite: reads back as NaN
    bad = x.copy()
    bad[3] = np.inf
    codes, scale, zero = kv4.quantise(bad)
    assert np.isnan(kv4.values(codes, scale, zero)).all()


@pytest.mark.parametrize("std", [1e-20, 1.0, 1e20])
def test_quantised_values_are_near(std):
    """Off by at most half a step, and by what rounding the scale (2^-8 of it,
    eight levels away) and the zero point (2^-8 of it) moves the levels."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 128)) * std).astype(np.float32)
    codes, scale, zero = kv4.quantise(x)
    s, z = (np.repeat(m.astype(np.float64), 64, -1) for m in (scale, zero))
    err = np.abs(kv4.values(codes, scale, zero) - x)
    assert (err <= s / 2 + 2.0 ** -8 * (16 * s + np.abs(z))).all()


def test_pack_order():
    codes = np.arange(16, dtype=np.uint8)[None]
    assert kv4.pack(codes)[0, :2].tolist() == [0x10, 0x32]
    np.testing.assert_array_equal(kv4.unpack(kv4.pack(codes)), codes)


def test_attention_of_the_last_token_equals_full_attention():
    rng = np.random.default_rng(2)
    B, S, H, Hk, D = 2, 37, 4, 2, 64
    q, k, v = rng.standard_normal((B, S, H, D)), rng.standard_normal((B, S, Hk, D)), rng.standard_normal((B, S, Hk, D))
    want, want_l = oracle.attention_naive(q, k, v, True, 0.125)
    out, lse, w = kv4.cache_attention(q[:, -3:], k.transpose(0, 2, 1, 3), v.transpose(0, 2, 1, 3),
                                      [S] * B, scale=0.125)
    np.testing.assert_allclose(out, want[:, -3:], atol=1e-12)
    np.testing.assert_allclose(lse, want_l[:, :, -3:], atol=1e-12)
    np.testing.assert_allclose(w.sum(-1), 3 * H // Hk, atol=1e-12)


def test_visible_by_definition():
    for p, n, w, k in itertools.product((-1, 0, 3, 9), (10,), (0, 1, 4, 99), (0, 2, 20)):
        want = [j <= p and (w == 0 or p - j < w or j < k) for j in range(n)]
        assert kv4.visible(p, n, w, k).tolist() == want


def test_evict_by_brute_force():
    rng = np.random.default_rng(3)
    for _ in range(200):
        n = int(rng.integers(1, 12))
        budget = int(rng.integers(1, 12))
        sink = int(rng.integers(0, budget + 1))
        recent = int(rng.integers(0, budget - sink + 1))
        score = rng.integers(0, 4, n).astype(np.float64)
        kept = kv4.evict(score, n, budget, sink, recent)
        assert kept == sorted(set(kept)) and len(kept) == min(n, budget)
        if n <= budget:
            continue
        assert set(range(sink)) <= set(kept) and set(range(n - recent, n)) <= set(kept)
        middle = [j for j in range(sink, n - recent)]
        for i in middle:
            for j in middle:
                better = score[i] > score[j] or (score[i] == score[j] and i < j)
                assert not (better and j in kept and i not in kept)
