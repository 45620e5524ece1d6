"""Sizes beyond 32 bits: the C ABI counts in int, and a Python integer keeps
its meaning on the way there instead of losing its upper bits."""

import sys

import pytest

from sequence_exact_attention_gb300 import binding

BIG = [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, sys.maxsize, 2 ** 70]


@pytest.mark.parametrize("big", BIG)
def test_a_window_or_first_tokens_past_the_end_mean_all_tokens(lib, big):
    sizes = (1, 8, 1, 3000, 128, 1)
    want = binding.bwd_window_workspace_bytes(*sizes, window=3000, n_sink=3000)
    few = binding.bwd_window_workspace_bytes(*sizes, window=5, n_sink=0)
    assert want != few
    assert binding.bwd_window_workspace_bytes(*sizes, window=big, n_sink=big) == want
    assert (binding.bwd_window_workspace_bytes(*sizes, window=5, n_sink=big) ==
            binding.bwd_window_workspace_bytes(*sizes, window=5, n_sink=3000) != few)
    cache = (2, 1, 8, 2, 128, 65536)
    none = binding.kv4_attn_workspace_bytes(*cache)
    assert none != binding.kv4_attn_workspace_bytes(*cache, window=300)
    assert binding.kv4_attn_workspace_bytes(*cache, window=big, n_sink=big) == none
    assert (binding.kv4_attn_workspace_bytes(*cache, window=300, n_sink=big) ==
            binding.kv4_attn_workspace_bytes(*cache, window=300, n_sink=65536))


@pytest.mark.parametrize("bad", [-1, -2 ** 31, -2 ** 32 + 5, -2 ** 70])
def test_negative_sizes_are_refused_whatever_their_lower_bits(lib, bad):
    sizes = (1, 8, 1, 3000, 128, 1)
    for kw in (dict(window=bad), dict(window=5, n_sink=bad)):
        with pytest.raises(binding.RingAttnError):
            binding.bwd_window_workspace_bytes(*sizes, **kw)
    cache = (2, 1, 8, 2, 128, 65536)
    for kw in (dict(window=bad), dict(window=5, n_sink=bad), dict(max_len=bad)):
        with pytest.raises(binding.RingAttnError):
            binding.kv4_attn_workspace_bytes(*cache, **kw)


@pytest.mark.parametrize("big", BIG)
def test_sizes_that_bound_others_are_refused_when_too_large(lib, big):
    with pytest.raises(binding.RingAttnError):
        binding.kv4_attn_workspace_bytes(2, 1, 8, 2, 128, 65536, max_len=big)
    with pytest.raises(binding.RingAttnError):              # 4 packed sequences of so many tokens
        binding.bwd_window_workspace_bytes(4, 8, 2, big, 128, 1, 100, varlen=True)
    with pytest.raises(binding.RingAttnError):
        binding.bwd_window_workspace_bytes(big, 8, 2, 100, 128, 1, 100)
