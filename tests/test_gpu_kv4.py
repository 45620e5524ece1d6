"""The 4-bit key/value cache (kv4_append, kv4_read, kv4_attn, kv4_evict)
against the NumPy oracle, through the C ABI.

Tolerances, from the arithmetic (u = half a step of the type, relative):
codes, scales, zero points and evicted rows are equal. A read value is one
float32 operation on exact inputs, rounded to the output type. A logit's error
E is at most (D + 8) 2^-23 of the sum of its absolute terms (products exact,
sums float32, the tensor core may drop the last bit of a term) and what small
query values lose in half precision: with the row's largest brought to 2^14 or
more and divided by at most 16, 2^-25 2^-10 of it, far less than the 2^-22
below, times the codes' values. A weight is then off by 2 E + 2^-21 (two
exponentials' errors) of itself, and its half-precision product with the value
scale by 2^-11 more, times the code's value less 8, that is |v - zero|; the
output is rounded to bf16 (2^-8).
"""

import numpy as np
import pytest
import torch

from oracle import kv4
from sequence_exact_attention_gb300 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


def random_cache(B, H, C, D, seed, junk_from=None):
    """(KV4Cache, k, v values [B, H, C, D] float64); slots from junk_from[b]
    on hold NaN metadata and arbitrary codes."""
    rng = np.random.default_rng(seed)
    parts, vals = [], []
    for _ in range(2):
        codes = rng.integers(0, 16, (B, H, C, D)).astype(np.uint8)
        scale = kv4.bf16((0.1 + rng.random((B, H, C, D // 64)) * 0.4).astype(np.float32))
        zero = kv4.bf16((0.3 * rng.standard_normal((B, H, C, D // 64))).astype(np.float32))
        vals.append(kv4.values(codes, scale, zero))
        meta = np.stack([scale, zero], -1)
        if junk_from is not None:
            for b in range(B):
                meta[b, :, max(0, junk_from[b]):] = np.nan
        parts += [torch.from_numpy(kv4.pack(codes)).to(DEV),
                  torch.from_numpy(meta).to(torch.bfloat16).to(DEV)]
    return binding.KV4Cache(*parts), vals[0], vals[1]


def bounds(q, k, v, lens, window, n_sink, out, scale):
    """(tolerance of out, of lse) from the module docstring's terms."""
    q = np.asarray(q, np.float64)
    B, S_q, H_q, D = q.shape
    grp = H_q // k.shape[1]
    t_out, t_lse = np.zeros(out.shape), np.zeros((B, H_q, S_q))
    for b in range(B):
        n = max(int(lens[b]), 0)
        for t in range(S_q):
            see = np.flatnonzero(kv4.visible(n - S_q + t, k.shape[2], window, n_sink)[:n])
            if see.size == 0:
                continue
            for h in range(H_q):
                kk, vv, qq = k[b, h // grp, see], v[b, h // grp, see], q[b, t, h]
                # |sk (c - 8)| + |zk| is at most 8 steps of 0.5 and a zero point below 1.5
                terms = 8.0 * np.abs(qq).sum()
                e = scale * ((D + 8) * 2.0 ** -23 * terms + 2.0 ** -24 * np.abs(qq).max() * D * 4.0)
                s = scale * (kk @ qq)
                p = np.exp(s - s.max())
                p /= p.sum()
                t_lse[b, h, t] = e + 2.0 ** -20 * (1 + np.abs(s).max())
                t_out[b, t, h] = (np.abs(out[b, t, h]) * 2.0 ** -8 +
                                  (2 * e + 2.0 ** -20 * (1 + np.abs(s).max()) + 2.0 ** -11) * (p @ (np.abs(vv) + 1.5)))
    return t_out, t_lse


def run_attn(q, cache, lens, C, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = binding.kv4_attn(q, cache, lens, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse


CASES = [
    # B, S_q, H_q, H_kv, D, C, lens, window, n_sink
    ("one_slot", 1, 1, 1, 1, 64, 16, [1], 0, 0),
    ("empty_and_full", 3, 1, 4, 2, 128, 64, [0, 64, 17], 0, 0),
    ("odd_lengths_gqa4", 4, 1, 16, 4, 128, 1040, [1033, 33, 512, 1], 0, 0),
    ("group_of_3", 2, 1, 6, 2, 64, 160, [159, 96], 0, 0),
    ("group_of_16", 1, 1, 32, 2, 128, 512, [500], 0, 0),
    ("group_of_20_two_blocks", 1, 1, 20, 1, 64, 96, [95], 0, 0),
    ("verify_4", 2, 4, 8, 2, 128, 208, [200, 7], 0, 0),
    ("verify_longer_than_the_sequence", 3, 5, 4, 4, 64, 48, [3, 5, 0], 0, 0),
    ("verify_7_of_group_8", 2, 7, 16, 2, 64, 320, [301, 64], 0, 0),
    ("window", 3, 1, 8, 2, 128, 1008, [1000, 100, 50], 100, 0),
    ("window_1", 2, 1, 4, 2, 64, 128, [128, 1], 1, 0),
    ("window_sink", 3, 3, 8, 2, 128, 2048, [2047, 300, 2], 130, 5),
    ("window_sink_many", 2, 1, 8, 8, 64, 4096, [4000, 2100], 65, 300),
    ("window_past_the_end", 1, 2, 4, 2, 128, 160, [150], 1 << 30, 4),
    ("long_split", 1, 1, 8, 2, 128, 20000, [19999], 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
@pytest.mark.parametrize("score", [False, True])
def test_attention_matches_oracle(case, score):
    _, B, S_q, H_q, H_kv, D, C, lens, window, n_sink = case
    cache, k, v = random_cache(B, H_kv, C, D, seed=B + C, junk_from=lens)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(B, S_q, H_q, D, generator=g).to(torch.bfloat16)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    before = torch.rand(B, H_kv, C, generator=g) * 3
    sc = before.to(DEV) if score else None
    out, lse = run_attn(q.to(DEV), cache, lens_d, C, window=window, n_sink=n_sink, score=sc)
    want, want_l, want_w = kv4.cache_attention(q, k, v, lens, window, n_sink)
    t_out, t_lse = bounds(q.float().numpy(), k, v, lens, window, n_sink, want, 1 / np.sqrt(D))
    got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(want_l)
    assert np.array_equal(np.isneginf(got_l), empty)
    assert np.all(np.abs(got - want) <= t_out), np.max(np.abs(got - want) - t_out)
    assert np.all(np.abs(got_l - want_l)[~empty] <= t_lse[~empty])
    if score:
        w = sc.double().cpu().numpy() - before.double().numpy()
        # each of the S_q * group weights within its bound, and the sum's rounding
        rel = 2 * t_lse.max() + 2.0 ** -20
        assert np.all(np.abs(w - want_w) <= rel * want_w + 2.0 ** -22 * (want_w + before.numpy()))
        assert np.array_equal(w[want_w == 0], np.zeros_like(w[want_w == 0]))


def test_masked_slots_may_hold_infinities():
    """Slots that the window hides hold NaN scales and infinite zero points."""
    B, H_q, H_kv, D, C = 1, 8, 2, 128, 512
    cache, k, v = random_cache(B, H_kv, C, D, seed=9)
    for meta in (cache.k_meta, cache.v_meta):
        meta[:, :, 4:380, :, 0] = float("nan")
        meta[:, :, 4:380, :, 1] = float("inf")
    q = torch.randn(B, 2, H_q, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    lens = torch.tensor([501], dtype=torch.int32, device=DEV)
    out, lse = run_attn(q.to(DEV), cache, lens, C, window=100, n_sink=4)
    want, want_l, _ = kv4.cache_attention(q, k, v, [501], 100, 4)
    t_out, t_lse = bounds(q.float().numpy(), k, v, [501], 100, 4, want, 1 / np.sqrt(D))
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= t_out)
    assert np.all(np.abs(lse.double().cpu().numpy() - want_l) <= t_lse)


def test_a_visible_nan_reaches_the_output():
    cache, _, _ = random_cache(1, 1, 64, 64, seed=3)
    cache.k_meta[0, 0, 5] = float("nan")
    q = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([40], dtype=torch.int32, device=DEV)
    out, lse = run_attn(q, cache, lens, 64)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    lens = torch.tensor([5], dtype=torch.int32, device=DEV)       # before it: finite
    out, lse = run_attn(q, cache, lens, 64)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("v_scale", [1e-30, 1e-6, 1e6, 1e30])
@pytest.mark.parametrize("q_scale", [1e-20, 1.0, 1e3])
def test_magnitudes(v_scale, q_scale):
    """Values and queries far from one: the power-of-two scalings hold."""
    B, H_q, H_kv, D, C, n = 1, 4, 2, 128, 256, 250
    cache, k, v = random_cache(B, H_kv, C, D, seed=11)
    f = float(torch.tensor(v_scale).to(torch.bfloat16))
    new = (cache.v_meta.float() * f).to(torch.bfloat16)
    cache = binding.KV4Cache(*cache[:3], new)
    v = kv4.values(kv4.unpack(cache.v_codes.cpu().numpy()), *(new.float().cpu().numpy()[..., i] for i in (0, 1)))
    q = (torch.randn(B, 1, H_q, D, generator=torch.Generator().manual_seed(2)) * q_scale).to(torch.bfloat16)
    scale = 1 / np.sqrt(D) / max(q_scale, 1.0)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    out, lse = run_attn(q.to(DEV), cache, lens, C, scale=scale)
    want, want_l, _ = kv4.cache_attention(q, k, v, [n], scale=scale)
    t_out, t_lse = bounds(q.float().numpy(), k, v / f, [n], 0, 0, want / f, scale)
    assert np.all(np.abs(out.double().cpu().numpy() - want) / f <= t_out)
    assert np.all(np.abs(lse.double().cpu().numpy() - want_l) <= t_lse)


def test_value_scales_that_grow_along_the_cache():
    """The largest value scale met so far rises tile by tile by 2^60."""
    B, H, D, C = 1, 2, 64, 512
    cache, k, v = random_cache(B, H, C, D, seed=12)
    growth = torch.exp2(torch.linspace(-30, 30, C).floor()).to(DEV)
    new = (cache.v_meta.float() * growth[None, None, :, None, None]).to(torch.bfloat16)
    cache = binding.KV4Cache(*cache[:3], new)
    v = kv4.values(kv4.unpack(cache.v_codes.cpu().numpy()), *(new.float().cpu().numpy()[..., i] for i in (0, 1)))
    q = torch.randn(B, 1, 2 * H, D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    for n in (512, 300, 40):
        lens = torch.tensor([n], dtype=torch.int32, device=DEV)
        out, _ = run_attn(q.to(DEV), cache, lens, C)
        want, _, _ = kv4.cache_attention(q, k, v, [n])
        top = np.abs(v[:, :, :n]).max()
        # the sum is dominated by the last slots: relative to its own terms
        t_out, _ = bounds(q.float().numpy(), k, v / top, [n], 0, 0, want / top, 1 / np.sqrt(D))
        assert np.all(np.abs(out.double().cpu().numpy() - want) / top <= t_out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,H,D,C", [(1, 1, 1, 64, 16), (3, 5, 2, 128, 64), (2, 33, 3, 64, 48)])
def test_append_and_read(dtype, B, T, H, D, C):
    rng = np.random.default_rng(B * 100 + T)
    k = torch.from_numpy((rng.standard_normal((B, T, H, D)) * 2).astype(np.float32)).to(dtype)
    v = torch.from_numpy((rng.standard_normal((B, T, H, D)) + 5).astype(np.float32)).to(dtype)
    k[0, 0, 0, :64] = 1.5                       # a constant group
    start = torch.tensor([(7 * b) % (C - T + 1) for b in range(B)], dtype=torch.int32, device=DEV)
    cache = binding.kv4_cache(B, H, C, D, DEV)
    for t in cache:
        t.fill_(3)
    before = [t.clone() for t in cache]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.kv4_append(cache, k.to(DEV), v.to(DEV), start, dev_status=status)
    for x, codes, meta, c0, m0 in ((k, *cache[:2], *before[:2]), (v, *cache[2:], *before[2:])):
        want_c, want_s, want_z = kv4.quantise(x.float().numpy())
        got_c, got_m = codes.cpu().numpy(), meta.float().cpu().numpy()
        for b in range(B):
            s0 = int(start[b])
            np.testing.assert_array_equal(got_c[b, :, s0:s0 + T], kv4.pack(want_c)[b].transpose(1, 0, 2))
            np.testing.assert_array_equal(got_m[b, :, s0:s0 + T, :, 0], want_s[b].transpose(1, 0, 2))
            np.testing.assert_array_equal(got_m[b, :, s0:s0 + T, :, 1], want_z[b].transpose(1, 0, 2))
            rest = [j for j in range(C) if not s0 <= j < s0 + T]
            assert torch.equal(codes[b, :, rest], c0[b, :, rest]) and torch.equal(meta[b, :, rest], m0[b, :, rest])
    rk, rv = binding.kv4_read(cache, start, T, dtype, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for got, x in ((rk, k), (rv, v)):
        want = kv4.values(*kv4.quantise(x.float().numpy()))
        u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= u * np.abs(want) + 2.0 ** -22)


def test_append_padding_and_slots_out_of_range():
    B, T, H, D, C = 3, 4, 1, 64, 16
    k = torch.randn(B, T, H, D, device=DEV)
    cache = binding.kv4_cache(B, H, C, D, DEV)
    start = torch.tensor([0, 14, -2], dtype=torch.int32, device=DEV)
    n_new = torch.tensor([2, 4, 4], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.kv4_append(cache, k, k, start, n_new=n_new, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 10                    # RA_ERR_RANGE: slots 16, 17 and -2, -1
    written = (cache.k_meta[:, 0, :, 0, 0] != 0).cpu()
    want = torch.zeros(B, C, dtype=torch.bool)
    want[0, :2] = want[1, 14:] = want[2, :2] = True
    assert torch.equal(written, want)
    status.zero_()
    rk, _ = binding.kv4_read(cache, start, T, torch.float32, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 10
    assert (rk[1, 2:] == 0).all() and (rk[2, :2] == 0).all() and (rk[2, 2:] != 0).any()


def test_not_finite_groups_read_as_nan():
    k = torch.randn(1, 3, 1, 128, device=DEV)
    k[0, 0, 0, 70] = float("inf")
    k[0, 1, 0, 3] = float("nan")
    cache = binding.kv4_cache(1, 1, 16, 128, DEV)
    binding.kv4_append(cache, k, k, torch.zeros(1, dtype=torch.int32, device=DEV))
    rk, _ = binding.kv4_read(cache, None, 3, torch.float32)
    nan = torch.isnan(rk)[0, :, 0].view(3, 2, 64)
    assert nan[0, 1].all() and nan[1, 0].all() and int(nan.sum()) == 128


EVICT = [
    # B, H, D, C, lens, budget, sink, recent
    ("one", 1, 1, 64, 16, [2], 1, 0, 0),
    ("nothing_to_evict", 2, 2, 128, 64, [10, 0], 16, 2, 3),
    ("mixed", 3, 2, 128, 400, [400, 100, 399], 112, 4, 30),
    ("all_protected", 1, 2, 64, 96, [90], 40, 10, 30),
    ("no_protection", 2, 1, 64, 1600, [1599, 77], 64, 0, 0),
    ("long", 1, 2, 64, 20000, [19990], 3000, 4, 500),
]


@pytest.mark.parametrize("kind", ["distinct", "ties", "special"])
@pytest.mark.parametrize("case", EVICT, ids=[c[0] for c in EVICT])
def test_evict_matches_oracle(case, kind):
    _, B, H, D, C, lens, budget, sink, recent = case
    cache, _, _ = random_cache(B, H, C, D, seed=C)
    rng = np.random.default_rng(C + budget)
    if kind == "distinct":
        score = np.exp(3 * rng.standard_normal((B, H, C))).astype(np.float32)
    elif kind == "ties":
        score = rng.integers(0, 3, (B, H, C)).astype(np.float32)
    else:
        score = rng.choice(np.array([np.nan, -np.inf, np.inf, -0.0, 0.0, 1e-40, -1e-40, -1.0, 2.0], np.float32),
                           (B, H, C))
    sd = torch.from_numpy(score).to(DEV)
    C_dst = -(-budget // 16) * 16 + 16
    dst = binding.kv4_cache(B, H, C_dst, D, DEV)
    for t in dst:
        t.fill_(7)
    ds = torch.full((B, H, C_dst), -5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    src = [t.clone() for t in cache]
    got, gs, gl, kept = binding.kv4_evict(cache, sd, torch.tensor(lens, dtype=torch.int32, device=DEV), budget, sink,
                                          recent, dst=dst, dst_score=ds, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert gl.tolist() == [min(n, budget) for n in lens]
    assert all(torch.equal(a, b) for a, b in zip(src, cache))
    for b in range(B):
        for h in range(H):
            want = kv4.evict(score[b, h], lens[b], budget, sink, recent)
            m = len(want)
            assert kept[b, h, :m].tolist() == want, (b, h)
            assert (kept[b, h, m:] == -1).all()
            for x, y in zip(cache, got):
                assert torch.equal(y[b, h, :m], x[b, h, want])
                assert (y[b, h, m:] == 7).all()
            np.testing.assert_array_equal(gs[b, h, :m].cpu().numpy(), score[b, h][want])
            assert (gs[b, h, m:] == -5).all()


def test_serving_loop_as_used():
    """Prompt, decoding, eviction, more decoding: append, attend with scores,
    evict, append again; every step against the oracle on the values that the
    cache holds. The steps run from one captured graph, on a side stream."""
    B, H_q, H_kv, D, C, budget = 2, 8, 2, 64, 96, 48
    g = torch.Generator().manual_seed(21)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)   # noqa: E731
    cache, spare = binding.kv4_cache(B, H_kv, C, D, DEV), binding.kv4_cache(B, H_kv, C, D, DEV)
    score = torch.zeros(B, H_kv, C, device=DEV)
    lens = torch.tensor([40, 23], dtype=torch.int32, device=DEV)
    binding.kv4_append(cache, rnd(B, 40, H_kv, D), rnd(B, 40, H_kv, D),
                       torch.zeros(B, dtype=torch.int32, device=DEV), n_new=lens)
    q, k, v = rnd(B, 1, H_q, D), rnd(B, 1, H_kv, D), rnd(B, 1, H_kv, D)
    ws = torch.empty(max(16, binding.kv4_attn_workspace_bytes(B, 1, H_q, H_kv, D, C, with_score=True)),
                     dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, H_q, 1, device=DEV)

    def step():
        binding.kv4_append(cache, k, v, lens)
        lens.add_(1)
        binding.kv4_attn(q, cache, lens, score=score, out=out, lse=lse, workspace=ws)

    def check(before):
        ks, vs = (kv4.values(kv4.unpack(c.cpu().numpy()), *(m.float().cpu().numpy()[..., i] for i in (0, 1)))
                  for c, m in (cache[:2], cache[2:]))
        want, want_l, w = kv4.cache_attention(q.cpu(), ks, vs, lens.tolist())
        t_out, t_lse = bounds(q.float().cpu().numpy(), ks, vs, lens.tolist(), 0, 0, want, 1 / np.sqrt(D))
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= t_out)
        assert np.all(np.abs(lse.double().cpu().numpy() - want_l) <= t_lse)
        got = (score - before).double().cpu().numpy()
        assert np.all(np.abs(got - w) <= 2.0 ** -18 * (w + 4))

    before = score.clone()
    step()
    torch.cuda.synchronize()
    check(before)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(12):
        for x in (q, k, v):
            x.copy_(rnd(*x.shape))
        before = score.clone()
        graph.replay()
        torch.cuda.synchronize()
        check(before)
    n = lens.tolist()
    assert n == [53, 36]
    _, s2, l2, kept = binding.kv4_evict(cache, score, lens, budget, 4, 16, dst=spare,
                                        dst_score=torch.zeros_like(score))
    for dst, src in ((cache, spare), ((score,), (s2,)), ((lens,), (l2,))):
        for a, b in zip(dst, src):
            a.copy_(b)                                     # the graph holds these buffers
    assert lens.tolist() == [48, 36] and kept.shape == (B, H_kv, budget)
    for x in (q, k, v):
        x.copy_(rnd(*x.shape))
    before = score.clone()
    graph.replay()
    torch.cuda.synchronize()
    check(before)


def test_calls_on_a_given_stream():
    """stream=: the launch and what the call allocates belong to it."""
    cache, k, v = random_cache(1, 2, 4096, 128, seed=31)
    q = torch.randn(1, 1, 8, 128, device=DEV).to(torch.bfloat16)
    lens = torch.tensor([4000], dtype=torch.int32, device=DEV)
    want, want_l = binding.kv4_attn(q, cache, lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = binding.kv4_attn(q, cache, lens, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_l)


def test_calls_side_by_side_and_from_two_graphs():
    """Attention with scores and eviction on two streams at once, eager and then
    as two captured graphs replayed together, equal the calls made alone."""
    torch.cuda.synchronize()
    work = []
    for seed in (61, 62):
        cache, _, _ = random_cache(2, 2, 4096, 64, seed=seed)
        q = torch.randn(2, 1, 8, 64, device=DEV).to(torch.bfloat16)
        lens = torch.tensor([4000, 2500 + seed], dtype=torch.int32, device=DEV)
        ws = torch.empty(binding.kv4_attn_workspace_bytes(2, 1, 8, 2, 64, 4096, with_score=True), dtype=torch.uint8,
                         device=DEV)
        work.append((cache, q, lens, torch.zeros(2, 2, 4096, device=DEV), ws, torch.cuda.Stream()))

    def step(cache, q, lens, score, ws, stream):
        score.zero_()
        out, lse = binding.kv4_attn(q, cache, lens, score=score, workspace=ws)
        dst, ds, dl, kept = binding.kv4_evict(cache, score, lens, 512, 4, 64)
        return (out, lse, score, ds, dl, kept, *dst)

    want = []
    for w in work:
        want.append([t.clone() for t in step(*w)])
        torch.cuda.synchronize()
    got = []
    for w in work:
        with torch.cuda.stream(w[-1]):
            got.append(step(*w))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    graphs = []
    for w in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=w[-1]):
            graphs.append((g, step(*w)))
    for _ in range(3):
        for (g, _), w in zip(graphs, work):
            with torch.cuda.stream(w[-1]):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for (_, x), y in zip(graphs, want) for a, b in zip(x, y))


def test_attention_repeats_bit_for_bit_and_merges():
    """Two halves of a cache merged by attn_lse_merge give the whole."""
    B, H_q, H_kv, D, C = 1, 8, 2, 128, 2048
    cache, _, _ = random_cache(B, H_kv, C, D, seed=41)
    q = torch.randn(B, 1, H_q, D, device=DEV).to(torch.bfloat16)
    n = lambda x: torch.tensor([x], dtype=torch.int32, device=DEV)     # noqa: E731
    out, lse = binding.kv4_attn(q, cache, n(2000))
    again, lse2 = binding.kv4_attn(q, cache, n(2000))
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    a, la = binding.kv4_attn(q, cache, n(1024))
    tail = binding.KV4Cache(*[t[:, :, 1024:].contiguous() for t in cache])
    b, lb = binding.kv4_attn(q, tail, n(976))
    m, lm = binding.attn_lse_merge(a, la, b, lb)
    # each side's bf16 rounding (2^-8 of it) and the merged one's
    tol = 2.0 ** -8 * (a.float().abs() + b.float().abs() + out.float().abs() + m.float().abs()) + 1e-3
    assert ((m.float() - out.float()).abs() <= tol).all()
    assert ((lm - lse).abs() <= 1e-5).all()


@pytest.fixture
def checked_library():
    prev = binding.use_library("debug")
    yield
    binding.use_library(prev)


def test_checked_build_is_in_range_and_identical(checked_library):
    def run(status):
        cache, _, _ = random_cache(2, 2, 1040, 128, seed=51)
        q = torch.randn(2, 3, 8, 128, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
        lens = torch.tensor([1033, 40], dtype=torch.int32, device=DEV)
        score = torch.zeros(2, 2, 1040, device=DEV)
        res = list(binding.kv4_attn(q, cache, lens, score=score, dev_status=status))
        res += list(binding.kv4_attn(q, cache, lens, window=77, n_sink=9, dev_status=status))
        binding.kv4_append(cache, q[:, :, :2].contiguous(), q[:, :, 2:4].contiguous(), lens - 3, dev_status=status)
        res += list(binding.kv4_read(cache, lens - 3, 3, dev_status=status))
        dst, s, n, kept = binding.kv4_evict(cache, score, lens, 100, 4, 30, dev_status=status)
        return res + [score, s, n, kept, *dst]

    binding.use_library("release")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = run(status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    binding.use_library("debug")
    got = run(status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
