"""4-bit cache attention of a chunk of a prompt: many new tokens at once over a
cache that already holds their context, far past the few of a decoding step."""

import numpy as np
import pytest
import torch

from oracle import kv4
from sequence_exact_attention_gb300 import binding

from test_gpu_kv4 import bounds, random_cache, run_attn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("B,S_q,H_q,H_kv,D,C,lens,window,n_sink", [
    (1, 33, 4, 2, 64, 640, [610], 0, 0),
    (2, 130, 8, 2, 128, 400, [390, 130], 0, 0),
    (1, 200, 3, 1, 64, 1040, [1033], 150, 5),
    (2, 100, 4, 4, 128, 512, [500, 40], 64, 3),       # the second sequence is shorter than its chunk
])
def test_chunk_of_a_prompt(B, S_q, H_q, H_kv, D, C, lens, window, n_sink, score):
    cache, k, v = random_cache(B, H_kv, C, D, seed=S_q, junk_from=lens)
    q = torch.randn(B, S_q, H_q, D, generator=torch.Generator().manual_seed(S_q)).to(torch.bfloat16)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    sc = torch.zeros(B, H_kv, C, device=DEV) if score else None
    out, lse = run_attn(q.to(DEV), cache, lens_d, C, window=window, n_sink=n_sink, score=sc)
    want, want_l, want_w = kv4.cache_attention(q, k, v, lens, window, n_sink)
    t_out, t_lse = bounds(q.float().numpy(), k, v, lens, window, n_sink, want, 1 / np.sqrt(D))
    got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(want_l)
    assert np.array_equal(np.isneginf(got_l), empty)
    assert np.all(np.abs(got - want) <= t_out)
    assert np.all(np.abs(got_l[~empty] - want_l[~empty]) <= t_lse[~empty])
    if score:
        # every weight within its bound, and the sum of as many as S_q * group of them
        rel = 2 * t_lse.max() + 2.0 ** -20 + S_q * (H_q // H_kv) * 2.0 ** -24
        w = sc.double().cpu().numpy()
        assert np.all(np.abs(w - want_w) <= rel * want_w)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (70, 4)])
def test_a_prompt_in_chunks_is_the_prompt_at_once(window, n_sink):
    """300 tokens appended and attended to in chunks of different sizes: rows,
    and scores, are those of one call over all of them."""
    H_q, H_kv, D, C, S = 8, 2, 64, 304, 300
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, S, h, D, generator=g).to(torch.bfloat16).to(DEV) for h in (H_q, H_kv, H_kv))
    whole, parts = (binding.kv4_cache(1, H_kv, C, D, DEV) for _ in range(2))
    at = lambda n: torch.tensor([n], dtype=torch.int32, device=DEV)      # noqa: E731
    s0, s1 = (torch.zeros(1, H_kv, C, device=DEV) for _ in range(2))
    binding.kv4_append(whole, k, v, at(0))
    want, want_l = binding.kv4_attn(q, whole, at(S), window=window, n_sink=n_sink, score=s0)
    n = 0
    for m in (1, 40, 2, 129, 128):
        binding.kv4_append(parts, k[:, n:n + m].contiguous(), v[:, n:n + m].contiguous(), at(n))
        out, lse = binding.kv4_attn(q[:, n:n + m].contiguous(), parts, at(n + m), window=window, n_sink=n_sink,
                                    score=s1)
        # blocks of rows and chunks of slots fall elsewhere: sums in another order, outputs rounded to bf16
        a, b = out.double(), want[:, n:n + m].double()
        assert ((a - b).abs() <= 2.0 ** -8 * (a.abs() + b.abs()) + 2.0 ** -10).all()
        assert ((lse - want_l[:, :, n:n + m]).abs() <= 2.0 ** -18 * (1 + lse.abs())).all()
        n += m
    assert n == S and all(torch.equal(a, b) for a, b in zip(whole, parts))
    # a slot's sum has at most S * 4 weights, each off by 2^-17 of itself, in another order
    assert ((s0 - s1).abs() <= (2.0 ** -16 + S * 4 * 2.0 ** -23) * s0).all()
