"""Pins of the paged cache's oracle (oracle/paged.py): the number format
against torch's, rows against hand values, pages against slot-by-slot loops,
attention against the full attention oracle."""

import numpy as np
import pytest
import torch

import oracle
from oracle import paged


def test_code_values_equal_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(paged.e4m3_values(), codes.double().numpy())


def test_hand_quantised_row():
    # 448 is the largest code: scale 1; 449 and more: scale 2
    x = np.zeros(64)
    x[:5] = [448.0, -17.0, 18.0, 19.0, 2.0 ** -10]
    codes, byte = paged.quantise(x)
    assert byte == 127
    # steps of 2 above 16: 17 is a tie and goes to the even mantissa (16), 19 to 20; 2^-10 is a tie with 0
    assert paged.values(codes, byte)[:5].tolist() == [448.0, -16.0, 18.0, 20.0, 0.0]
    x[0] = 449.0
    codes, byte = paged.quantise(x)
    assert byte == 128 and paged.values(codes, byte)[0] == 448.0
    assert paged.quantise(np.zeros(64))[1] == 10          # nothing to scale: the least
    x[1], x[2] = np.inf, np.nan
    codes, byte = paged.quantise(x)
    assert byte == 128 and np.isnan(paged.values(codes, byte)[1:3]).all()
    assert paged.values(codes, byte)[3] == 20.0


@pytest.mark.parametrize("std", [1e-30, 1.0, 1e30])
def test_codes_equal_torchs_conversion(std):
    x = (np.random.default_rng(1).standard_normal((32, 128)) * std).astype(np.float32)
    codes, byte = paged.quantise(x)
    y = torch.from_numpy(x.astype(np.float64) / 2.0 ** (byte.astype(np.float64) - 127)[:, None])
    assert float(y.abs().max()) <= 448 and float(y.abs().amax(-1).min()) > 224
    np.testing.assert_array_equal(codes, y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    # off by at most half a step: 2^-4 of the value, or of the least normal one, 2^-6
    got = paged.values(codes, byte)
    step = 2.0 ** (byte.astype(np.float64) - 127)[:, None]
    assert np.all(np.abs(got - x) <= 2.0 ** -4 * np.maximum(np.abs(x), 2.0 ** -6 * step))


def test_slots_are_found_in_their_pages():
    pool = np.arange(5 * 2 * 16 * 3).reshape(5, 2, 16, 3)
    table = np.array([[3, 0], [-1, 4], [5, 2]])
    got, has = paged.rows(pool, table, 40), paged.there(table, 5, 16, 40)
    for b in range(3):
        for j in range(40):
            ok = j < 32 and 0 <= table[b, j // 16] < 5
            assert has[b, j] == ok
            if ok:
                np.testing.assert_array_equal(got[b, :, j], pool[table[b, j // 16], :, j % 16])


def test_a_whole_prompt_is_causal_attention():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((1, 20, h, 64)) for h in (4, 2, 2))
    kk, vv = (np.moveaxis(x, 1, 2) for x in (k, v))
    out, lse = paged.attention([q[0]], kk, vv, [20], [20], np.ones((1, 20), bool))
    want, want_l = oracle.attention_naive(q, k, v, True, 0.125)
    np.testing.assert_allclose(out[0], want[0], atol=1e-12)
    np.testing.assert_allclose(lse[0], want_l[0], atol=1e-12)
    # its last five tokens alone, behind the first fifteen; a page that is not there
    out, lse = paged.attention([q[0, 15:]], kk, vv, [20], [5], np.ones((1, 20), bool))
    np.testing.assert_allclose(out[0], want[0, 15:], atol=1e-12)
    has = np.ones((1, 20), bool)
    has[0, :16] = False
    out, lse = paged.attention([q[0, 15:]], kk, vv, [20], [5], has)
    assert np.all(np.isneginf(lse[0][:, 0])) and np.all(out[0][0] == 0)
    np.testing.assert_allclose(out[0][1], v[0, 16].repeat(2, 0), atol=1e-12)
