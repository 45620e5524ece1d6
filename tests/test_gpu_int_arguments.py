"""Sizes beyond 32 bits in calls: a window or a count past the end means all
tokens, a bound that no size can reach is refused."""

import sys

import pytest
import torch

from sequence_exact_attention_gb300 import binding

from test_gpu_kv4 import random_cache

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


@pytest.mark.parametrize("big", [2 ** 32 + 5, 2 ** 32, sys.maxsize])
def test_windowed_attention(big):
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(1, 300, h, 64, generator=g).to(torch.bfloat16).to(DEV) for h in (4, 2, 2, 4))
    cu = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    for window, n_sink in ((big, 0), (5, big), (big, big)):
        small = [min(x, 300) for x in (window, n_sink)]
        res = []
        for w in ((window, n_sink), small):
            out, lse = binding.ring_attn_fwd_window(q, k, v, 1, *w)
            r = [out, lse, *binding.ring_attn_bwd_window(q, k, v, out, lse, do, 1, *w)]
            out, lse = binding.ring_attn_fwd_window_varlen(q[0], k[0], v[0], cu, 300, 1, *w)
            r += [out, lse, *binding.ring_attn_bwd_window_varlen(q[0], k[0], v[0], out, lse, do[0], cu, 300, 1, *w)]
            res.append(r)
        assert all(torch.equal(a, b) for a, b in zip(*res))
    for bad in (dict(window=-big), dict(window=5, n_sink=-big)):
        with pytest.raises(binding.RingAttnError):
            binding.ring_attn_fwd_window(q, k, v, 1, **bad)
    with pytest.raises(binding.RingAttnError):
        binding.ring_attn_fwd_window_varlen(q[0], k[0], v[0], cu, big, 1, 5)


@pytest.mark.parametrize("big", [2 ** 32 + 5, 2 ** 32 + 16, sys.maxsize])
def test_cache(big):
    cache, _, _ = random_cache(1, 2, 128, 64, seed=2)
    q = torch.randn(1, 1, 4, 64, device=DEV).to(torch.bfloat16)
    lens = torch.tensor([120], dtype=torch.int32, device=DEV)
    for kw, small in ((dict(window=big), dict()), (dict(window=9, n_sink=big), dict(window=9, n_sink=128)),
                      (dict(window=big, n_sink=big), dict())):
        for a, b in zip(binding.kv4_attn(q, cache, lens, **kw), binding.kv4_attn(q, cache, lens, **small)):
            assert torch.equal(a, b)
    score = torch.zeros(1, 2, 128, device=DEV)
    dst = binding.kv4_cache(1, 2, 128, 64, DEV)
    for call in (lambda: binding.kv4_attn(q, cache, lens, max_len=big),
                 lambda: binding.kv4_evict(cache, score, lens, 64, big),
                 lambda: binding.kv4_evict(cache, score, lens, 64, 0, big),
                 lambda: binding.kv4_evict(cache, score, lens, 64, 0, -big),
                 lambda: binding.kv4_evict(cache, score, lens, big), lambda: binding.kv4_evict(cache, score, lens, -big),
                 lambda: binding.kv4_evict(cache, score, lens, big, dst=dst)):
        with pytest.raises((binding.RingAttnError, ValueError)):
            call()
