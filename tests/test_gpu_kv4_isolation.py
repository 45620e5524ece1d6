"""4-bit cache attention: what a query does not see changes nothing of its
results, and values far larger than the others cost those no precision.

The cache holds ordinary values but for one slot, whose value scale and zero
point are ordinary, 2^30 times larger, infinite or not a number. Tolerances are
those of tests/test_gpu_kv4.py with the terms of a value v = scale (c - 8) +
zero written out: a weight p_j is off by its logit's error E_j, the weighted mean
of all E and 2^-20 (1 + max |s|) of itself, its half-precision product w_j = p_j scale_j by 2^-11 more, or, where that is a
subnormal half, by half its step 2^-25. A row's products of a group are
multiplied by a power of two that keeps the largest met so far at 1 or more, so
that is at most 2^-25 of the group's largest w (allowed: twice that), each of n
visible slots' |c - 8| <= 8 times over. The output is rounded to bf16 (2^-8 of itself).
"""

import numpy as np
import pytest
import torch

from oracle import kv4
from sequence_exact_attention_gb300 import binding

from test_gpu_kv4 import random_cache, run_attn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
INF, NAN = float("inf"), float("nan")


def host(cache):
    """Keys, their scales and zero points, and the values' three, float64 [B, H, C, D]."""
    parts = []
    for codes, meta in (cache[:2], cache[2:]):
        m = meta.double().cpu().numpy()
        scale, zero = (np.repeat(m[..., i], 64, -1) for i in (0, 1))
        with np.errstate(invalid="ignore"):
            parts.append((scale * (kv4.unpack(codes.cpu().numpy()).astype(np.float64) - 8) + zero, scale, zero))
    return [x for p in parts for x in p]


def expected(q, cache, lens, window=0, n_sink=0, scale=None):
    """(out, its bound, lse, its bound), float64, row by row from the visible slots alone."""
    k, sk, zk, v, sv, zv = host(cache)
    q = q.double().cpu().numpy()
    B, S_q, H_q, D = q.shape
    grp = H_q // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, t_out = np.zeros(q.shape), np.zeros(q.shape)
    lse, t_lse = np.full((B, H_q, S_q), -np.inf), np.zeros((B, H_q, S_q))
    for b in range(B):
        n = int(lens[b])
        for t in range(S_q):
            see = np.flatnonzero(kv4.visible(n - S_q + t, k.shape[2], window, n_sink)[:max(n, 0)])
            if see.size == 0:
                continue
            for h in range(H_q):
                kk, ks, kz, vv, ss, zz = (x[b, h // grp, see] for x in (k, sk, zk, v, sv, zv))
                qq = q[b, t, h]
                s = scale * (kk @ qq)
                p = np.exp(s - s.max())
                total = p.sum()
                p /= total
                # of the logits' terms |q| |sk (c - 8)| + |q| |zk|, and the codes' of |q| in halves, as there
                e = scale * ((D + 8) * 2.0 ** -23 * ((8 * np.abs(ks) + np.abs(kz)) @ np.abs(qq)) +
                             2.0 ** -24 * np.abs(qq).max() * 8 * np.abs(ks).sum(1))
                more = 2.0 ** -20 * (1 + np.abs(s).max())
                weight = p * (e + p @ e + more + 2.0 ** -11)
                with np.errstate(invalid="ignore"):
                    out[b, t, h] = p @ vv
                    terms = weight @ (np.abs(vv - zz) + np.abs(zz))
                    lost = see.size * 8 * 2.0 ** -24 * np.max(p[:, None] * np.abs(ss), axis=0)
                    t_out[b, t, h] = 2.0 ** -8 * np.abs(out[b, t, h]) + terms + lost
                lse[b, h, t] = s.max() + np.log(total)
                t_lse[b, h, t] = p @ e + more
    return out, t_out, lse, t_lse


def with_values(cache, at, factor, groups=slice(None)):
    """The cache with slot `at`'s value scales and zero points (of some groups) times factor."""
    meta = cache.v_meta.clone()
    meta[:, :, at, groups] = (meta[:, :, at, groups].float() * factor).to(torch.bfloat16)
    return binding.KV4Cache(*cache[:3], meta)


def queries(B, S_q, H_q, D, seed):
    return torch.randn(B, S_q, H_q, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def inside(got, want, tol):
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), np.max(err - tol)


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("D,grp,n", [(64, 1, 20), (128, 2, 200), (128, 4, 77), (64, 8, 5000)])
def test_a_later_tokens_values_leave_earlier_tokens_alone(D, grp, n, score):
    """Four drafted tokens; the last one's values are of any size or kind."""
    S_q, H_kv, C = 4, 2, -(-n // 16) * 16
    plain, _, _ = random_cache(1, H_kv, C, D, seed=n, junk_from=[n])
    q = queries(1, S_q, H_kv * grp, D, 3)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    first = None
    for factor in (1.0, 2.0 ** 30, -2.0 ** 60, INF, NAN):
        cache = with_values(plain, n - 1, factor)
        sc = torch.zeros(1, H_kv, C, device=DEV) if score else None
        out, lse = run_attn(q.to(DEV), cache, lens, C, score=sc)
        want, t_out, want_l, t_lse = expected(q, cache, [n])
        inside(lse, want_l, t_lse)
        inside(out[:, :3], want[:, :3], t_out[:, :3])
        if np.isfinite(factor):
            inside(out[:, 3:], want[:, 3:], t_out[:, 3:])
        else:
            assert not torch.isfinite(out[:, 3]).any()
        got = [out[:, :3], lse] + ([sc] if score else [])
        first = [t.clone() for t in got] if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("D,grp,n,window,n_sink", [(64, 1, 300, 100, 0), (128, 2, 1000, 130, 5), (128, 4, 45, 20, 2)])
def test_a_slot_that_left_the_window_is_left_alone(D, grp, n, window, n_sink):
    """Only the first of four tokens still sees the slot."""
    S_q, H_kv, C = 4, 2, -(-n // 16) * 16
    at = n - S_q - window + 1
    plain, _, _ = random_cache(1, H_kv, C, D, seed=n + 1)
    q = queries(1, S_q, H_kv * grp, D, 4)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    first = None
    for factor in (1.0, 2.0 ** 30, INF, NAN):
        cache = with_values(plain, at, factor)
        out, lse = run_attn(q.to(DEV), cache, lens, C, window=window, n_sink=n_sink)
        want, t_out, want_l, t_lse = expected(q, cache, [n], window, n_sink)
        inside(lse, want_l, t_lse)
        inside(out[:, 1:], want[:, 1:], t_out[:, 1:])
        if np.isfinite(factor):
            inside(out[:, :1], want[:, :1], t_out[:, :1])
        else:
            assert not torch.isfinite(out[:, 0]).any()
        got = [out[:, 1:], lse]
        first = [t.clone() for t in got] if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_an_infinite_draft_that_was_appended():
    """As it comes about: a drafted token with one infinite value in one group."""
    B, S_q, H_q, H_kv, D, n, C = 2, 3, 8, 2, 128, 150, 160
    plain, _, _ = random_cache(B, H_kv, C, D, seed=8)
    lens = torch.tensor([n, 90], dtype=torch.int32, device=DEV)
    q, k, v = queries(B, S_q, H_q, D, 5), queries(B, S_q, H_kv, D, 6), queries(B, S_q, H_kv, D, 7)
    v[1, 2, 0, 70] = INF                     # second group of the last token, first key/value head
    binding.kv4_append(plain, k.to(DEV), v.to(DEV), lens - S_q)
    out, lse = run_attn(q.to(DEV), plain, lens, C)
    want, t_out, want_l, t_lse = expected(q, plain, lens.tolist())
    inside(lse, want_l, t_lse)
    bad = np.isnan(want)
    assert bad.sum() == 4 * 64 and bad[1, 2, :4, 64:].all()
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), bad)
    assert np.all(np.abs(got - want)[~bad] <= t_out[~bad])


@pytest.mark.parametrize("D,S_q", [(64, 1), (128, 1), (128, 4)])
@pytest.mark.parametrize("at", [slice(0, 1), slice(57, 58), slice(140, 141), slice(299, 300), slice(0, 32),
                                slice(120, 180)], ids=lambda s: f"{s.start}to{s.stop}")
def test_large_values_of_small_weight(D, S_q, at):
    """Visible slots with values 2^40 times the others' and weights far below
    2^-60: the others' share of the output keeps its precision, wherever those
    slots come."""
    H_kv, C, n = 2, 320, 300
    cache, _, _ = random_cache(1, H_kv, C, D, seed=13)
    codes, meta = cache.k_codes.clone(), cache.k_meta.clone()
    codes[:, :, at] = 0x88                   # the same key value everywhere, the queries' sum far below 0
    meta[:, :, at, :, 1] = 64 / D ** 0.5
    cache = with_values(binding.KV4Cache(codes, meta, *cache[2:]), at, 2.0 ** 40)
    q = queries(1, S_q, 4, D, 9) - 1.0
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    out, lse = run_attn(q.to(DEV), cache, lens, C)
    want, t_out, want_l, t_lse = expected(q, cache, [n])
    plain, _, _, _ = expected(q, with_values(cache, at, 2.0 ** -40), [n])
    assert np.all(np.abs(want - plain) <= 2.0 ** -20)      # they count for next to nothing
    inside(out, want, t_out)
    inside(lse, want_l, t_lse)


@pytest.mark.parametrize("factor", [2.0 ** 40, 2.0 ** -40])
@pytest.mark.parametrize("score", [False, True])
def test_groups_of_different_size(factor, score):
    """One group of 64 dimensions far larger or smaller than the other."""
    H_kv, D, C, n = 2, 128, 400, 390
    cache, _, _ = random_cache(1, H_kv, C, D, seed=14)
    cache = with_values(cache, slice(None), factor, groups=0)
    q = queries(1, 2, 8, D, 10)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    sc = torch.zeros(1, H_kv, C, device=DEV) if score else None
    out, lse = run_attn(q.to(DEV), cache, lens, C, score=sc)
    want, t_out, want_l, t_lse = expected(q, cache, [n])
    inside(out, want, t_out)
    inside(lse, want_l, t_lse)


def test_scales_below_zero():
    """A cache made elsewhere may hold negative scales."""
    H_kv, D, C, n = 2, 64, 272, 260
    cache, _, _ = random_cache(1, H_kv, C, D, seed=15)
    parts = list(cache)
    for i in (1, 3):
        parts[i] = parts[i].clone()
        parts[i][:, :, ::3, :, 0] *= -1
    parts[3][:, :, 100:, :, 0] *= 2.0 ** 20
    cache = binding.KV4Cache(*parts)
    q = queries(1, 1, 4, D, 11)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    out, lse = run_attn(q.to(DEV), cache, lens, C)
    want, t_out, want_l, t_lse = expected(q, cache, [n])
    inside(out, want, t_out)
    inside(lse, want_l, t_lse)


@pytest.mark.parametrize("D,S_q", [(64, 1), (128, 3)])
@pytest.mark.parametrize("growth", [0.2, 1.0])
def test_scores_that_grow_over_values_of_all_sizes(D, S_q, growth):
    """Every tile raises the running maxima, by `growth` a slot, and value scales
    lie anywhere between 2^-30 and 2^30 of the others': the largest product so far
    is an old one in one row, a new one in another."""
    H_kv, C, n = 2, 640, 630
    cache, _, _ = random_cache(1, H_kv, C, D, seed=16)
    rng = np.random.default_rng(17)
    parts = [t.clone() for t in cache]
    slope = torch.arange(C, device=DEV) * (growth / D ** 0.5)
    parts[1][..., 1] = slope[None, None, :, None].to(torch.bfloat16)
    size = torch.from_numpy(2.0 ** rng.integers(-30, 31, (1, H_kv, C, D // 64, 1))).to(DEV)
    parts[3] = (parts[3].double() * size).to(torch.bfloat16)
    cache = binding.KV4Cache(*parts)
    q = queries(1, S_q, 4, D, 18) * 0.25 + 1.0
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    out, lse = run_attn(q.to(DEV), cache, lens, C)
    want, t_out, want_l, t_lse = expected(q, cache, [n])
    inside(out, want, t_out)
    inside(lse, want_l, t_lse)
