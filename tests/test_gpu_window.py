"""Windowed attention with first tokens that stay visible (ring_attn_fwd_window,
ring_attn_bwd_window and their packed forms) against the float64 oracle.

Tolerances are those of the entry points beside them, from the same
arithmetic: bf16 forward 2e-2 / 2e-3 (max / mean, tests/helpers.py), float32
1e-4, gradients 2e-2 of the largest and 1e-2 of the mean reference entry
(tests/test_gpu_backward.py).
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import kv4
from sequence_exact_attention_gb300 import binding

from helpers import assert_close

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


def rel(got, want):
    d = np.abs(got.detach().double().cpu().numpy() - want)
    return d.max() / max(np.abs(want).max(), 1e-2), d.mean() / max(np.abs(want).mean(), 1e-2)


def check_grads(got, want):
    for name, g, w in zip(("dq", "dk", "dv"), got, want):
        mx, mean = rel(g, w)
        assert np.isfinite(mx) and mx <= 2e-2 and mean <= 1e-2, (name, mx, mean)


def draw(rows, H_q, H_kv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*rows, h, D, generator=g).to(dtype) for h in (H_q, H_kv, H_kv, H_q)]


CASES = [
    # name, B, H_q, H_kv, S, D, P, order, window, n_sink
    ("s1", 1, 2, 1, 1, 64, 1, "contiguous", 1, 0),
    ("s130_w1", 2, 2, 2, 130, 128, 1, "contiguous", 1, 0),
    ("s130_w1_sink1", 1, 2, 1, 130, 64, 1, "contiguous", 1, 1),
    ("s777_w100_sink7", 2, 4, 2, 777, 64, 1, "contiguous", 100, 7),
    ("s1024_w128", 1, 2, 2, 1024, 128, 1, "contiguous", 128, 0),
    ("s1024_w129_sink128", 1, 4, 1, 1024, 128, 2, "zigzag", 129, 128),
    ("s1500_w257_sink129_zigzag", 1, 2, 2, 1500, 128, 3, "zigzag", 257, 129),
    ("s1001_w64_sink4_p8", 1, 4, 2, 1001, 64, 8, "zigzag", 64, 4),
    ("s900_w300_sink400", 1, 2, 1, 900, 128, 1, "contiguous", 300, 400),
    ("s5_mostly_empty", 1, 2, 1, 5, 64, 4, "contiguous", 2, 1),
    ("s3000_w500_sink16_gqa4", 1, 8, 2, 3000, 64, 1, "contiguous", 500, 16),
    ("s1100_w40_sink32", 1, 2, 1, 1100, 128, 1, "contiguous", 40, 32),
    ("s1100_w200_sink33", 1, 2, 1, 1100, 64, 2, "zigzag", 200, 33),
    ("s1300_w130_sink160", 1, 2, 2, 1300, 64, 1, "contiguous", 130, 160),
    ("s1301_w256_sink161_p2", 1, 2, 2, 1301, 128, 2, "contiguous", 256, 161),
    ("s1300_w600_sink20_p5", 1, 2, 2, 1300, 128, 5, "zigzag", 600, 20),
    ("s1500_mqa7_heads_shared", 1, 7, 1, 1500, 128, 1, "contiguous", 300, 0),
    ("s700_gqa6_heads_and_positions_shared", 2, 12, 2, 700, 64, 1, "contiguous", 90, 140),
    ("window_past_the_end", 1, 2, 2, 300, 128, 1, "contiguous", 1 << 30, 1 << 30),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matches_oracle(case, dtype):
    _, B, H_q, H_kv, S, D, P, order, window, n_sink = case
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, do = draw((B, S), H_q, H_kv, D, tdt, 100 + S)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    qd, kd, vd, dd = (t.to(DEV) for t in (q, k, v, do))
    out, lse = binding.ring_attn_fwd_window(qd, kd, vd, P, window, n_sink, order=order, dev_status=status)
    scale = 1 / np.sqrt(D)
    want, want_l = oracle.window_attention(q, k, v, window, n_sink, scale)
    assert_close(out, want, dtype, "out")
    assert_close(lse, want_l, dtype, "lse")
    if dtype == "bf16":
        got = binding.ring_attn_bwd_window(qd, kd, vd, out, lse, dd, P, window, n_sink, order=order,
                                           dev_status=status)
        check_grads(got, oracle.window_backward(q, k, v, do, window, n_sink, scale))
    torch.cuda.synchronize()
    assert int(status.item()) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,n_sink", [(2, 0), (3, 1), (1, 1), (7, 4), (16, 0), (300, 0)])
def test_gradients_lose_no_more_than_two_roundings(D, window, n_sink):
    """dq and dk come from dS in bf16 and are rounded to it: two roundings of
    one size, sqrt(2) times the error of rounding the exact gradient, and a
    tenth for everything else. Rows of few keys lose no more (they would, with
    delta from the rounded output)."""
    q, k, v, do = draw((1, 1000), 4, 2, D, torch.bfloat16, 77)
    qd, kd, vd, dd = (t.to(DEV) for t in (q, k, v, do))
    out, lse = binding.ring_attn_fwd_window(qd, kd, vd, 1, window, n_sink)
    got = binding.ring_attn_bwd_window(qd, kd, vd, out, lse, dd, 1, window, n_sink)
    want = oracle.window_backward(q, k, v, do, window, n_sink, 1 / np.sqrt(D))
    for name, g, w in zip(("dq", "dk", "dv"), got, want):
        rounded = torch.from_numpy(w).to(torch.bfloat16).double().numpy()
        err = np.linalg.norm(g.double().cpu().numpy() - w)
        assert err <= 1.1 * np.sqrt(2) * np.linalg.norm(rounded - w), (name, err / np.linalg.norm(w))


@pytest.mark.parametrize("lengths,D", [([5, 2, 16, 1, 9, 12] * 20, 64), ([61, 15], 128), ([16, 1, 38, 11, 58], 64),
                                       ([33, 40, 70] * 3, 128)])
def test_packed_sequences_of_few_tokens(lengths, D):
    """No row sees more than its short sequence: the same holds."""
    total, longest = sum(lengths), max(lengths)
    q, k, v, do = draw((total,), 4, 2, D, torch.bfloat16, 78)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cud = torch.from_numpy(cu).to(DEV)
    qd, kd, vd, dd = (t.to(DEV) for t in (q, k, v, do))
    out, lse = binding.ring_attn_fwd_window_varlen(qd, kd, vd, cud, longest, 1, 100, 4)
    got = binding.ring_attn_bwd_window_varlen(qd, kd, vd, out, lse, dd, cud, longest, 1, 100, 4)
    want = oracle.window_backward_varlen(q, k, v, do, cu, 100, 4, 1 / np.sqrt(D))
    for name, g, w in zip(("dq", "dk", "dv"), got, want):
        rounded = torch.from_numpy(w).to(torch.bfloat16).double().numpy()
        err = np.linalg.norm(g.double().cpu().numpy() - w)
        assert err <= 1.1 * np.sqrt(2) * np.linalg.norm(rounded - w), (name, err / np.linalg.norm(w))


PACKED = [
    # lengths, H_q, H_kv, D, P, order, window, n_sink
    ("mixed", [300, 0, 1, 777, 128, 1000], 4, 2, 128, 1, "contiguous", 100, 4),
    ("mixed_zigzag", [300, 0, 1, 777, 128, 1000], 4, 2, 64, 4, "zigzag", 130, 150),
    ("long_and_short", [2500, 3, 40], 2, 1, 64, 1, "contiguous", 64, 16),
    ("mqa8_heads_shared", [700, 0, 130, 5], 8, 1, 64, 1, "contiguous", 200, 9),
    ("one_token_each", [1, 1, 1], 2, 2, 128, 2, "contiguous", 1, 1),
]


@pytest.mark.parametrize("case", PACKED, ids=[c[0] for c in PACKED])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_matches_oracle(case, dtype):
    _, lengths, H_q, H_kv, D, P, order, window, n_sink = case
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    total, longest = sum(lengths), max(lengths)
    pad = 7                                            # rows behind the last sequence
    q, k, v, do = draw((total + pad,), H_q, H_kv, D, tdt, 200 + total)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cud = torch.from_numpy(cu).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    qd, kd, vd, dd = (t.to(DEV) for t in (q, k, v, do))
    out = torch.full_like(qd, 7.0)
    lse = torch.full((H_q, total + pad), 7.0, device=DEV)
    binding.ring_attn_fwd_window_varlen(qd, kd, vd, cud, longest, P, window, n_sink, order=order, out=out, lse=lse,
                                        dev_status=status)
    scale = 1 / np.sqrt(D)
    real = [t[:total] for t in (q, k, v, do)]
    want, want_l = oracle.window_attention_varlen(*real[:3], cu, window, n_sink, scale)
    assert_close(out[:total], want, dtype, "out")
    assert_close(lse[:, :total], want_l, dtype, "lse")
    assert (out[total:] == 7).all() and (lse[:, total:] == 7).all()
    if dtype == "bf16":
        grads = [torch.full_like(t, 7.0) for t in (qd, kd, vd)]
        got = binding.ring_attn_bwd_window_varlen(qd, kd, vd, out, lse, dd, cud, longest, P, window, n_sink,
                                                  order=order, dq=grads[0], dk=grads[1], dv=grads[2],
                                                  dev_status=status)
        check_grads([g[:total] for g in got], oracle.window_backward_varlen(*real, cu, window, n_sink, scale))
        assert all((g[total:] == 7).all() for g in got)
    torch.cuda.synchronize()
    assert int(status.item()) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_window_over_everything_is_the_causal_call(D, dtype):
    # a query head a key/value head: no heads are shared out, which would change the order of sums
    q, k, v, do = (t.to(DEV) for t in draw((1, 700), 4, 4, D, dtype, 31))
    a, la = binding.ring_attn_fwd(q, k, v, 1, True)
    for P, order in ((1, "contiguous"), (2, "zigzag"), (8, "contiguous")):
        b, lb = binding.ring_attn_fwd_window(q, k, v, P, 700, 0, order=order)
        if dtype == torch.float32:
            # two kernels that sum in different orders, each within 1e-4 of the
            # definition and far nearer here
            assert_close(b, a.cpu().numpy(), "f32", "out")
            assert_close(lb, la.cpu().numpy(), "f32", "lse")
        else:
            # the same sums in the same order, whatever the ranks
            assert torch.equal(a, b) and torch.equal(la, lb)
            want = binding.ring_attn_bwd(q, k, v, a, la, do, 1, True)
            got = binding.ring_attn_bwd_window(q, k, v, b, lb, do, P, 700, 0, order=order)
            # but for the first 32 rows' delta, which windowed calls do not take from the rounded
            # output: those rows of dq, and all of dk, may differ by what that rounding is worth,
            # which is less than the half step 2^-8 that either result is rounded by
            assert torch.equal(want[2], got[2]) and torch.equal(want[0][:, 32:], got[0][:, 32:])
            for x, y in zip(want[:2], got[:2]):
                assert (x.double() - y.double()).norm() <= 2.0 ** -8 * x.double().norm()
            first = got if P == 1 else first
            assert all(torch.equal(x, y) for x, y in zip(got, first))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,order", [(1, "contiguous"), (2, "zigzag")])
def test_packed_sequences_do_not_leak(D, dtype, P, order):
    """NaN and infinities in one sequence, and in the rows behind the last one,
    stay there: the others' results keep their bits."""
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lengths, pad, W, K = [300, 130, 77, 5], 140, 60, 6
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cud, rows = torch.from_numpy(cu).to(DEV), int(cu[-1]) + pad
    clean = [t.to(DEV) for t in draw((rows,), 4, 2, D, tdt, 71)]
    res = []
    for junk in (False, True):
        q, k, v, do = (t.clone() for t in clean)
        if junk:
            for t, x, y in ((q, np.nan, -np.inf), (k, np.inf, np.nan), (v, np.nan, np.inf), (do, np.inf, np.nan)):
                t[cu[1]:cu[2]] = x
                t[cu[-1]:] = y
        out, lse = torch.zeros_like(q), torch.zeros(4, rows, device=DEV)
        binding.ring_attn_fwd_window_varlen(q, k, v, cud, 300, P, W, K, order=order, out=out, lse=lse)
        got = [out, lse.t()]
        if dtype == "bf16":
            grads = [torch.zeros_like(t) for t in (q, k, v)]
            got += binding.ring_attn_bwd_window_varlen(q, k, v, out, lse, do, cud, 300, P, W, K, order=order,
                                                       dq=grads[0], dk=grads[1], dv=grads[2])
        res.append(got)
    for a, b in zip(*res):
        for lo, hi in ((cu[0], cu[1]), (cu[2], cu[3]), (cu[3], cu[4]), (cu[4], rows)):
            assert torch.equal(a[lo:hi], b[lo:hi])


@pytest.mark.parametrize("n_sink", [4, 200])
def test_gradients_repeat_and_ignore_the_workspace(n_sink):
    """Split shares of the first tokens' tiles: bit for bit the same with any
    workspace contents, and every gradient row is written."""
    q, k, v, do = (t.to(DEV) for t in draw((2, 4000), 4, 1, 128, torch.bfloat16, 32))
    out, lse = binding.ring_attn_fwd_window(q, k, v, 1, 200, n_sink)
    need = binding.bwd_window_workspace_bytes(2, 4, 1, 4000, 128, 1, 200, n_sink)
    assert need > binding.bwd_workspace_bytes(2, 4, 4000, 128, 1)         # parts to join
    res = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
        res.append(binding.ring_attn_bwd_window(q, k, v, out, lse, do, 1, 200, n_sink, dq=dq, dk=dk, dv=dv,
                                                workspace=ws))
    for a, b in zip(*res):
        assert torch.equal(a, b) and torch.isfinite(a).all()


def test_hidden_rows_may_hold_anything_large():
    """Keys that no window reaches any more do not move later rows."""
    S, W = 1200, 128
    q, k, v, _ = draw((1, S), 2, 2, 128, torch.bfloat16, 33)
    a, la = binding.ring_attn_fwd_window(*(t.to(DEV) for t in (q, k, v)), 1, W, 3)
    k2, v2 = k.clone(), v.clone()
    k2[:, 3:600] = 3e38
    v2[:, 3:600] = -3e38
    b, lb = binding.ring_attn_fwd_window(*(t.to(DEV) for t in (q, k2, v2)), 1, W, 3)
    first = 600 + W
    assert torch.equal(a[:, first:], b[:, first:]) and torch.equal(la[:, :, first:], lb[:, :, first:])


def test_captured_step_and_a_given_stream():
    """Forward and backward replayed from a graph, on new inputs, equal the
    eager calls; two graphs with their own workspaces replay side by side."""
    S, H, D, W, K = 900, 4, 64, 150, 5
    graphs = []
    for seed in (1, 2):
        q, k, v, do = (t.to(DEV) for t in draw((1, S), H, 2, D, torch.bfloat16, seed))
        out, lse = torch.empty_like(q), torch.empty(1, H, S, device=DEV)
        grads = [torch.empty_like(t) for t in (q, k, v)]
        ws = torch.empty(binding.bwd_window_workspace_bytes(1, H, 2, S, D, 1, W, K), dtype=torch.uint8, device=DEV)

        def step(q=q, k=k, v=v, do=do, out=out, lse=lse, grads=grads, ws=ws):
            binding.ring_attn_fwd_window(q, k, v, 1, W, K, out=out, lse=lse)
            binding.ring_attn_bwd_window(q, k, v, out, lse, do, 1, W, K, dq=grads[0], dk=grads[1], dv=grads[2],
                                         workspace=ws)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, (q, k, v, do), (out, lse, *grads)))
    for _, ins, _ in graphs:
        for t in ins:
            t.copy_(torch.randn(t.shape).to(t.dtype))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, (g, _, _) in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for s, (_, (q, k, v, do), got) in zip(streams, graphs):
        out, lse = binding.ring_attn_fwd_window(q, k, v, 1, W, K, stream=s)
        want = (out, lse, *binding.ring_attn_bwd_window(q, k, v, out, lse, do, 1, W, K, stream=s))
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_prompt_then_decoding_as_used():
    """A windowed prompt, its keys and values appended to a 4-bit cache, then
    decoding steps under the same window and first tokens; the prompt's first
    tokens and the steps are checked against the oracles."""
    B, S, H_q, H_kv, D, W, K, C = 2, 500, 8, 2, 128, 90, 4, 512
    q, k, v, _ = draw((B, S), H_q, H_kv, D, torch.bfloat16, 41)
    qd, kd, vd = (t.to(DEV) for t in (q, k, v))
    out, lse = binding.ring_attn_fwd_window(qd, kd, vd, 1, W, K)
    want, want_l = oracle.window_attention(q, k, v, W, K, 1 / np.sqrt(D))
    assert_close(out, want, "bf16", "prompt")
    cache = binding.kv4_cache(B, H_kv, C, D, DEV)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    binding.kv4_append(cache, kd, vd, zero)
    rk, rv = binding.kv4_read(cache, zero, S)
    for r, x in ((rk, k), (rv, v)):
        step = (x.float().view(B, S, H_kv, 2, 64).amax(-1) - x.float().view(B, S, H_kv, 2, 64).amin(-1)) / 15
        err = (r.cpu().float() - x.float()).abs().view(B, S, H_kv, 2, 64).amax(-1)
        # half a step, the level's move by rounding scale and zero, the output's rounding
        assert (err <= 0.5 * step + 2.0 ** -8 * (16 * step + 2 * x.float().abs().max())).all()
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    for i in range(3):
        nq, nk, nv, _ = (t.to(DEV) for t in draw((B, 1), H_q, H_kv, D, torch.bfloat16, 50 + i))
        binding.kv4_append(cache, nk, nv, lens)
        lens = lens + 1
        o, l = binding.kv4_attn(nq, cache, lens, window=W, n_sink=K)
        vals = [kv4.values(kv4.unpack(c.cpu().numpy()), *(m.float().cpu().numpy()[..., j] for j in (0, 1)))
                for c, m in (cache[:2], cache[2:])]
        w, wl, _ = kv4.cache_attention(nq.cpu(), *vals, lens.tolist(), W, K)
        assert_close(o, w, "bf16", "step")
        assert_close(l, wl, "bf16", "lse")


@pytest.fixture
def checked_library():
    prev = binding.use_library("debug")
    yield
    binding.use_library(prev)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_checked_build_is_in_range_and_identical(checked_library, dtype):
    def run(status):
        res = []
        for P, order, W, K in ((1, "contiguous", 100, 5), (4, "zigzag", 60, 300)):
            q, k, v, do = (t.to(DEV) for t in draw((1, 1001), 4, 2, 128, dtype, 61))
            out, lse = binding.ring_attn_fwd_window(q, k, v, P, W, K, order=order, dev_status=status)
            res += [out, lse]
            if dtype == torch.bfloat16:
                res += binding.ring_attn_bwd_window(q, k, v, out, lse, do, P, W, K, order=order, dev_status=status)
            lengths = [300, 0, 1, 700]
            cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
            out, lse = binding.ring_attn_fwd_window_varlen(q[0], k[0], v[0], cu, 700, P, W, K, order=order,
                                                           dev_status=status)
            res += [out, lse]
            if dtype == torch.bfloat16:
                res += [g[:1001] for g in binding.ring_attn_bwd_window_varlen(
                    q[0], k[0], v[0], out, lse, do[0], cu, 700, P, W, K, order=order, dev_status=status)]
        return res

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
