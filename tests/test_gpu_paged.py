"""The paged key/value cache (paged_append, paged_read, paged_attn and their
packed forms) against the NumPy oracle, through the C ABI.

Tolerances, from the arithmetic (u = half a step of the type, relative):
codes, scales and read values are equal. A logit's error E is at most
(D + 8) 2^-23 of the sum of its absolute terms (products exact, sums float32,
the tensor core may drop the last bit of a term); 8-bit pages: scales are powers
of two, and what small query values lose in half precision, 2^-24 of a quantum
where the row's largest is 2^14 or more, is far below that. A weight is then off
by 2 E + 2^-20 (1 + |s|) of itself (exponentials) and by its rounding, 2^-8 for
bf16 (bf16 pages, and packed pieces longer than a few rows), 2^-11 for half; sums
of n terms add n 2^-24; the output is rounded to bf16 (2^-8).
"""

import numpy as np
import pytest
import torch

from oracle import paged
from sequence_exact_attention_gb300 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
E4M3 = torch.float8_e4m3fn
RANGE = 10


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pool:
    """A pool with a table: sequences' pages in no order, a few spare ones, and
    everything that no slot in use holds filled with NaN."""

    def __init__(self, kind, H, page, D, lens, width, seed, spare=3):
        rng = np.random.default_rng(seed)
        held = [-(-max(n, 0) // page) for n in lens]
        self.n = sum(held) + spare
        ids = rng.permutation(self.n)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.shape = (self.n, H, page, D)
        used = np.zeros((self.n, page), bool)
        for b, n in enumerate(lens):
            for j in range(max(n, 0)):
                used[self.table[b, j // page], j % page] = True
        self.used = used
        parts = []
        if kind == "bf16":
            self.values = []
            for _ in range(2):
                x = torch.from_numpy(rng.standard_normal(self.shape).astype(np.float32)).to(torch.bfloat16)
                x[torch.from_numpy(~used)[:, None].expand(-1, H, -1)] = float("nan")
                self.values.append(x.double().numpy())
                parts.append(x.to(DEV))
        else:
            codes, scales, self.values = [], [], []
            for _ in range(2):
                c = rng.integers(0, 126, self.shape).astype(np.uint8) | (rng.integers(0, 2, self.shape) << 7).astype(np.uint8)
                e = rng.integers(117, 121, self.shape[:3]).astype(np.uint8)
                c[np.broadcast_to(~used[:, None], self.shape[:3])] = 127
                e[np.broadcast_to(~used[:, None], self.shape[:3])] = 254
                self.values.append(paged.values(c, e))
                codes.append(torch.from_numpy(c).to(DEV).view(E4M3))
                scales.append(torch.from_numpy(e).to(DEV))
            parts = codes + scales
        self.cache = binding.PagedCache(*parts)
        self.table_d = torch.from_numpy(self.table).to(DEV)

    def rows(self, n):
        """k, v [B, H, n, D] and which slots are there [B, n]."""
        k, v = (paged.rows(x, self.table, n) for x in self.values)
        return k, v, paged.there(self.table, self.n, self.shape[2], n)


def bounds(q, k, v, lens, news, has, window, n_sink, outs, u_w, scale):
    """Tolerances of out and of lse, sequence by sequence."""
    t_outs, t_lses = [], []
    for b, x in enumerate(q):
        x = np.asarray(x, np.float64)
        n_b, H_q, D = x.shape
        grp = H_q // k.shape[1]
        t_out, t_lse = np.zeros(x.shape), np.zeros((H_q, n_b))
        for t in range(n_b):
            p = int(lens[b]) - int(news[b]) + t
            j = np.arange(k.shape[2])
            see = (j <= p) & has[b]
            if window > 0:
                see &= (j > p - window) | (j < n_sink)
            see = np.flatnonzero(see)
            if see.size == 0:
                continue
            for h in range(H_q):
                kk, vv = k[b, h // grp, see], v[b, h // grp, see]
                e = scale * (D + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(x[t, h])).max()
                s = scale * (kk @ x[t, h])
                w = np.exp(s - s.max())
                w /= w.sum()
                rel = 2 * e + 2.0 ** -20 * (1 + np.abs(s).max()) + see.size * 2.0 ** -24
                t_lse[h, t] = rel
                t_out[t, h] = np.abs(outs[b][t, h]) * 2.0 ** -8 + (rel + u_w) * (w @ np.abs(vv))
        t_outs.append(t_out)
        t_lses.append(t_lse)
    return t_outs, t_lses


CASES = [
    # name, lens, new tokens of each (equal: also as a batch), H_q, H_kv, D, page, width, window, n_sink
    ("one_slot", [1], [1], 1, 1, 64, 16, 1, 0, 0),
    ("empty_and_full", [0, 64, 17], [1, 1, 1], 4, 2, 128, 16, 4, 0, 0),
    ("odd_lengths_gqa4", [1033, 33, 512, 1], [1, 1, 1, 1], 16, 4, 128, 32, 33, 0, 0),
    ("group_of_3", [159, 96], [1, 1], 6, 2, 64, 32, 5, 0, 0),
    ("group_of_16_page128", [500], [1], 32, 2, 128, 128, 4, 0, 0),
    ("group_of_20_two_blocks", [95], [1], 20, 1, 64, 16, 6, 0, 0),
    ("verify_4", [200, 7], [4, 4], 8, 2, 128, 64, 4, 0, 0),
    ("verify_longer_than_the_sequence", [3, 5, 0], [5, 5, 5], 4, 4, 64, 16, 3, 0, 0),
    ("verify_7_of_group_8", [301, 64], [7, 7], 16, 2, 64, 64, 5, 0, 0),
    ("window", [1000, 100, 50], [1, 1, 1], 8, 2, 128, 16, 63, 100, 0),
    ("window_1", [128, 1], [1, 1], 4, 2, 64, 16, 8, 1, 0),
    ("window_sink", [2047, 300, 3], [3, 3, 3], 8, 2, 128, 128, 16, 130, 5),
    ("window_sink_many", [4000, 2100], [1, 1], 8, 8, 64, 64, 64, 65, 300),
    ("window_past_the_end", [150], [2], 4, 2, 128, 32, 5, 1 << 30, 4),
    ("long_split", [19999], [1], 8, 2, 128, 64, 313, 0, 0),
    ("long_split_batch", [9000, 12, 4097], [2, 2, 2], 8, 1, 64, 16, 563, 0, 0),
    ("pieces", [33, 0, 200, 77, 1], [33, 0, 5, 1, 1], 4, 2, 64, 16, 13, 0, 0),
    ("pieces_gqa8_window", [140, 300, 64], [17, 140, 64], 8, 1, 128, 32, 10, 50, 3),
    ("piece_behind_a_prefix", [700], [130], 2, 2, 64, 64, 11, 0, 0),
    ("piece_group_5", [300, 290], [61, 200], 10, 2, 128, 16, 19, 0, 0),
    ("prompt_tiles", [640, 257], [640, 257], 4, 4, 64, 128, 5, 0, 0),
    ("prompt_few_rows_long", [6000], [40], 4, 1, 128, 128, 47, 0, 0),
    ("prompt_window_d128", [900, 520], [400, 520], 4, 2, 128, 64, 15, 200, 10),
    ("several_blocks_of_few_rows", [515, 40, 129], [5, 5, 5], 18, 2, 128, 16, 33, 0, 0),
    ("several_blocks_window", [515, 40, 300], [3, 1, 12], 8, 2, 64, 64, 9, 70, 3),
    ("group_of_128", [70, 3], [1, 1], 128, 1, 64, 16, 5, 0, 0),
    ("group_of_100", [70, 40], [3, 2], 100, 1, 128, 32, 3, 0, 0),
    ("a_wide_table", [300, 129, 40], [200, 1, 40], 4, 2, 64, 16, 20000, 0, 0),
    ("many_sequences", [3 * i % 50 for i in range(70)], [(3 * i % 50) * (i % 3) // 2 for i in range(70)], 2, 1, 64, 16, 4, 0,
     0),
    # wide tables: short and long ones in two launches over 8-bit pages
    ("short_beside_long", [900, 1, 64, 700, 0, 2, 33, 17, 500, 1], [1, 1, 4, 300, 0, 2, 1, 17, 5, 1], 8, 2, 128, 16, 1000, 0, 0),
    ("short_beside_long_window", [15000, 131, 64, 15900, 5, 222, 330, 177, 129], [3, 5, 6, 30, 5, 2, 1, 10, 7], 12, 4, 64, 64,
     250, 14500, 300),
    ("short_beside_long_split", [5000, 4999, 1, 4097, 130, 3000, 64, 2049], [1, 2, 1, 60, 1, 1, 4, 1], 4, 1, 128, 128, 260, 0, 0),
    ("short_beside_long_group_of_20", [300, 40, 200, 129, 7, 64, 90, 1], [1, 1, 100, 2, 1, 3, 1, 1], 20, 1, 64, 32, 2048, 0, 0),
    ("short_beside_one_of_30", [60 + i for i in range(40)], [1] * 39 + [30], 16, 2, 128, 16, 240, 0, 0),
    ("none_of_them_long", [3 * i for i in range(12)], [0, 1, 1, 2, 1, 0, 1, 2, 1, 1, 1, 1], 8, 2, 64, 16, 3, 0, 0),
    ("many_single_tokens", [7 * i % 90 for i in range(67)], [1] * 67, 2, 2, 64, 32, 3, 20, 1),
]


def check(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    inf = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), inf), what
    off = np.abs(got[~inf] - want[~inf]) - tol[~inf]
    assert np.all(off <= 0), (what, float(off.max()))     # (a NaN is not <= 0)


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_matches_oracle(case, kind):
    _, lens, news, H_q, H_kv, D, page, width, window, n_sink = case
    pool = Pool(kind, H_kv, page, D, lens, width, seed=sum(lens) + D)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(sum(news), H_q, D, generator=g).to(torch.bfloat16)
    parts = list(torch.split(q.float(), news))
    n = max(max(lens), 1)
    k, v, has = pool.rows(n)
    k, v = np.nan_to_num(k), np.nan_to_num(v)
    want, want_l = paged.attention([x.numpy() for x in parts], k, v, lens, news, has, window, n_sink)
    # bf16 weights also where 8-bit pages meet whole tiles of rows
    u_w = 2.0 ** -8 if kind == "bf16" or max(news) * H_q // H_kv > 16 else 2.0 ** -11
    t_out, t_lse = bounds([x.numpy() for x in parts], k, v, lens, news, has, window, n_sink, want, u_w, D ** -0.5)
    st = status_word()
    cu = ints(np.concatenate([[0], np.cumsum(news)]).tolist())
    # three rows behind the last sequence stay as they were
    qp = torch.cat([q, torch.full((3, H_q, D), float("nan"), dtype=q.dtype)]).to(DEV)
    out = torch.full_like(qp, 7.0)
    lse = torch.full((H_q, sum(news) + 3), 7.0, device=DEV)
    binding.paged_attn_varlen(qp, pool.cache, pool.table_d, ints(lens), cu, max(news), window=window, n_sink=n_sink, out=out,
                              lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool((out[-3:] == 7).all()) and bool((lse[:, -3:] == 7).all())
    at = 0
    for b, x in enumerate(news):
        check(out[at:at + x], want[b], t_out[b], f"out of {b}")
        check(lse[:, at:at + x], want_l[b], t_lse[b], f"lse of {b}")
        at += x
    if len(set(news)) == 1:
        B, T = len(news), news[0]
        out1, lse1 = binding.paged_attn(q.view(B, T, H_q, D).to(DEV), pool.cache, pool.table_d, ints(lens), window=window,
                                        n_sink=n_sink, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert torch.equal(out1.view(-1, H_q, D), out[:-3])
        assert torch.equal(lse1.transpose(0, 1).reshape(H_q, -1), lse[:, :-3])


def odd_rows(shape, dtype, seed):
    """Rows with zeros, the smallest and largest numbers, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-20, 20, shape[:-1], generator=g).float())[..., None]
    flat = x.view(-1, shape[-1])
    flat[0] = 0.0
    if flat.shape[0] > 6:
        flat[1] *= 1e-38
        flat[2] = 0.0
        flat[2, 3] = -1e-40
        flat[3, :] = 0.0
        flat[3, 5] = 3e38
        flat[4, 1], flat[4, 2], flat[4, 7] = float("inf"), float("-inf"), float("nan")
        flat[5] = float("nan")
        flat[6, :2] = torch.tensor([448.0, 449.0]) * 2.0 ** 10
    return x.to(dtype)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,page,H", [(64, 16, 3), (128, 64, 2)])
@pytest.mark.parametrize("packed", [False, True])
def test_append_and_read(kind, dtype, D, page, H, packed):
    starts, news, width = [0, 5, 37, 2 * page], [13, 0, page + 9, 1], 1 + (37 + 9) // page + 2
    B, T = 4, max(news)
    lens = [s + n for s, n in zip(starts, news)]
    pool = Pool(kind, H, page, D, lens, width, seed=3)
    before = [t.clone().view(torch.uint8) for t in pool.cache]
    st = status_word()
    if packed:
        k, v = (odd_rows((sum(news) + 2, H, D), dtype, s) for s in (1, 2))
        fresh = [list(torch.split(x[:-2], news)) for x in (k, v)]
        cu = ints(np.concatenate([[0], np.cumsum(news)]).tolist())
        binding.paged_append_varlen(pool.cache, pool.table_d, k.to(DEV), v.to(DEV), cu, ints(starts), dev_status=st)
    else:
        k, v = (odd_rows((B, T, H, D), dtype, s) for s in (1, 2))
        fresh = [[x[b, :n] for b, n in enumerate(news)] for x in (k, v)]
        binding.paged_append(pool.cache, pool.table_d, k.to(DEV), v.to(DEV), ints(starts), n_new=ints(news), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # what the pool has to hold now, element by element
    want = [t.cpu().clone() for t in before]
    for i in range(2):
        full = want[i].view(torch.bfloat16 if kind == "bf16" else torch.uint8)
        for b, n in enumerate(news):
            for t in range(n):
                at, row = pool.table[b, (starts[b] + t) // page], (starts[b] + t) % page
                x = fresh[i][b][t]
                if kind == "bf16":
                    full[at, :, row] = x.to(torch.bfloat16)
                else:
                    c, e = paged.quantise(x.double().numpy())
                    full[at, :, row] = torch.from_numpy(c)
                    want[2 + i][at, :, row] = torch.from_numpy(e)
    for name, x, y in zip(("k", "v", "k_scale", "v_scale"), pool.cache, want):
        x = x.view(torch.uint8).cpu()
        if kind == "bf16":          # NaN may have any bits
            a, b = x.view(torch.bfloat16), y.view(torch.bfloat16)
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num()), name
        else:
            assert torch.equal(x, y), name
    # read back, from before the new tokens to behind the last page
    first = [max(0, s - 2) for s in starts]
    n = width * page + 3
    got = binding.paged_read(pool.cache, pool.table_d, ints(first), n, dtype=dtype)
    parts = [t.cpu() for t in pool.cache]
    if kind == "bf16":
        held = [t.double().numpy() for t in parts]
    else:
        held = [paged.values(t.view(torch.uint8).numpy(), e.numpy()) for t, e in zip(parts[:2], parts[2:])]
    ok = paged.there(pool.table, pool.n, page, n + max(first))
    for x, pool_values in zip(got, held):
        all_rows = paged.rows(pool_values, pool.table, n + max(first))
        for b in range(B):
            y = np.moveaxis(all_rows[b, :, first[b]:first[b] + n], 0, 1)
            y = np.where(ok[b, first[b]:first[b] + n, None, None], y, 0.0)
            y = torch.from_numpy(y).to(dtype)
            z = x[b].cpu()
            assert torch.equal(z.isnan(), y.isnan()) and torch.equal(z.nan_to_num(), y.nan_to_num())


def test_slots_without_a_page():
    """Appended nowhere, read as zeros, not attended to; each says so."""
    for kind in ("bf16", "e4m3"):
        pool = Pool(kind, 2, 16, 64, [80], 6, seed=4)
        gone = pool.table.copy()
        gone[0, 1], gone[0, 3] = -1, pool.n
        table = torch.from_numpy(gone).to(DEV)
        x = torch.randn(1, 80, 2, 64, device=DEV).to(torch.bfloat16)
        before = [t.clone() for t in pool.cache]
        st = status_word()
        binding.paged_append(pool.cache, table, x[:, :70], x[:, :70], ints([30]), dev_status=st)
        assert int(st.item()) == RANGE                      # slots 30, 31, 48-63 and from 80 on
        for t, old in zip(pool.cache, before):
            for page in (pool.table[0, 1], pool.table[0, 3]):
                assert torch.equal(t[page].view(torch.uint8), old[page].view(torch.uint8))
            t.view(torch.uint8).copy_(old.view(torch.uint8))
        st.zero_()
        k, v = binding.paged_read(pool.cache, table, None, 80, dev_status=st)
        assert int(st.item()) == RANGE
        kk, vv = (np.moveaxis(r, 1, 2) for r in pool.rows(80)[:2])
        hole = np.zeros(80, bool)
        hole[16:32] = hole[48:64] = True
        for got, want in ((k, kk), (v, vv)):
            np.testing.assert_array_equal(got[0].double().cpu().numpy(), np.where(hole[:, None, None], 0, want[0]))
        for n_new in (1, 2, 40):                            # few rows, two positions, whole tiles of rows
            q = torch.randn(1, n_new, 4, 64, device=DEV).to(torch.bfloat16)
            st.zero_()
            out, lse = binding.paged_attn(q, pool.cache, table, ints([80]), dev_status=st)
            assert int(st.item()) == RANGE
            k64, v64, _ = pool.rows(80)
            qn = [q[0].float().cpu().numpy()]
            want, want_l = paged.attention(qn, k64, v64, [80], [n_new], ~hole[None])
            t_out, t_lse = bounds(qn, k64, v64, [80], [n_new], ~hole[None], 0, 0, want, 2.0 ** -8, 0.125)
            check(out[0], want[0], t_out[0], "out")
            check(lse[0], want_l[0], t_lse[0], "lse")
        # a window that has left the holes behind does not meet them
        st.zero_()
        q = torch.randn(1, 1, 4, 64, device=DEV).to(torch.bfloat16)
        binding.paged_attn(q, pool.cache, table, ints([80]), window=16, dev_status=st)
        assert int(st.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 4, 10])
def test_a_row_is_not_touched_by_what_it_does_not_see(kind, group):
    """A later drafted token's keys and values that are not finite change no
    bit of the rows before it; slots that a window hides none of any."""
    H, D = 2, 128
    pool = Pool(kind, H, 32, D, [150], 5, seed=6)
    q = torch.randn(1, 4, H * group, D, device=DEV).to(torch.bfloat16)
    out, lse = binding.paged_attn(q, pool.cache, pool.table_d, ints([150]), window=60, n_sink=2)
    at, row = pool.table[0, 148 // 32], 148 % 32            # the third new token
    far = pool.table[0, 1]                                  # slots 32 to 63: behind every window
    for t in pool.cache[:2]:
        bad = 0x7f if kind == "e4m3" else float("inf")
        raw = t.view(torch.uint8) if kind == "e4m3" else t
        raw[at, :, row, ::3] = bad
        raw[far] = bad
    got, got_l = binding.paged_attn(q, pool.cache, pool.table_d, ints([150]), window=60, n_sink=2)
    assert torch.equal(got[:, :2], out[:, :2]) and torch.equal(got_l[:, :, :2], lse[:, :, :2])
    assert bool(got[:, 2:].isnan().any())


def test_decoding_continues_the_forward():
    """A prompt through ring_attn_fwd, its keys and values appended in pieces,
    then token by token: every step equals the forward of the whole sequence,
    and a piece over its own slots merges with the prefix's."""
    H_q, H_kv, D, S, P = 8, 2, 128, 300, 260
    g = torch.Generator(device=DEV).manual_seed(8)
    q, k, v = (torch.randn(1, S, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (H_q, H_kv, H_kv))
    want, want_l = binding.ring_attn_fwd(q, k, v, 1, True)
    cache = binding.paged_cache(24, H_kv, 16, D)
    table = torch.randperm(24, generator=g, device=DEV).int()[None, :20].contiguous()

    def near(x, y, xl, yl):
        # both sides round weights and outputs to bf16, 2^-8 each of values of some 1
        assert float((x.float() - y.float()).abs().max()) <= 2 * 2.0 ** -8 * float(v.float().abs().max())
        assert float((xl - yl).abs().max()) <= 1e-5

    for lo, hi in ((0, 130), (130, 131), (131, P)):
        start, lens = ints([lo]), ints([hi])
        binding.paged_append(cache, table, k[:, lo:hi].contiguous(), v[:, lo:hi].contiguous(), start)
        out, lse = binding.paged_attn(q[:, lo:hi].contiguous(), cache, table, lens)
        near(out, want[:, lo:hi], lse, want_l[:, :, lo:hi])
    lens, start = ints([P + 1]), ints([P])
    for s in range(P, S):
        binding.paged_append(cache, table, k[:, s:s + 1].contiguous(), v[:, s:s + 1].contiguous(), start)
        out, lse = binding.paged_attn(q[:, s:s + 1].contiguous(), cache, table, lens)
        near(out, want[:, s:s + 1], lse, want_l[:, :, s:s + 1])
        start += 1
        lens += 1
    back = binding.paged_read(cache, table, None, S)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)
    # the prefix (no new token sees itself) and the piece alone, merged
    lo = 200
    piece = q[:, lo:P].contiguous()
    o1, l1 = binding.ring_attn_fwd(piece, k[:, lo:P].contiguous(), v[:, lo:P].contiguous(), 1, True)
    one = torch.cat([piece.view(-1, 1, H_q, D)])            # every token a sequence of its own over the prefix
    o0, l0 = binding.paged_attn(one, cache, table.expand(P - lo, 20).contiguous(), ints([lo] * (P - lo)))
    o, l = binding.attn_lse_merge(o0.view(1, -1, H_q, D), l0[:, :, 0].t().contiguous()[None], o1, l1)
    near(o, want[:, lo:P], l, want_l[:, :, lo:P])


def test_sequences_that_share_pages():
    """A prefix's pages in two tables: both sequences read them."""
    pool = Pool("bf16", 2, 32, 64, [96, 40], 4, seed=10)
    table = pool.table.copy()
    table[1, :3] = table[0, :3]
    q = torch.randn(1, 1, 4, 64, device=DEV).to(torch.bfloat16).expand(2, 1, 4, 64).contiguous()
    out, lse = binding.paged_attn(q, pool.cache, torch.from_numpy(table).to(DEV), ints([96, 96]))
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])


@pytest.mark.parametrize("n_new", [1, 40])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_step_replays_while_it_grows(kind, n_new):
    """Append, attention and their workspaces in a graph; lengths, tables and
    tokens change between replays. A second graph with a workspace of its own
    runs beside it on another stream."""
    H_q, H_kv, D, page, width = 8, 2, 128, 16, 300
    cap = page * width
    g = torch.Generator(device=DEV).manual_seed(1)
    make = lambda h: torch.randn(2, n_new, h, D, generator=g, device=DEV).to(torch.bfloat16)    # noqa: E731
    sides = []
    for _ in range(2):
        cache = binding.paged_cache(2 * width, H_kv, page, D, dtype=torch.bfloat16 if kind == "bf16" else E4M3)
        fill = torch.randn(2, cap, H_kv, D, generator=g, device=DEV).to(torch.bfloat16)
        table = torch.randperm(2 * width, generator=g, device=DEV).int().view(2, width)
        binding.paged_append(cache, table, fill, fill, ints([0, 0]))
        ws = torch.empty(binding.paged_attn_workspace_bytes(cache, 2, n_new, H_q, cap) + 16, dtype=torch.uint8, device=DEV)
        sides.append({"cache": cache, "table": table, "q": make(H_q), "k": make(H_kv), "v": make(H_kv),
                      "start": ints([100, 3000]), "lens": ints([100 + n_new, 3000 + n_new]),
                      "out": torch.empty(2, n_new, H_q, D, dtype=torch.bfloat16, device=DEV),
                      "lse": torch.empty(2, H_q, n_new, device=DEV), "ws": ws})

    def step(s):
        binding.paged_append(s["cache"], s["table"], s["k"], s["v"], s["start"])
        binding.paged_attn(s["q"], s["cache"], s["table"], s["lens"], out=s["out"], lse=s["lse"], workspace=s["ws"])

    graphs = []
    for s in sides:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(s)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(s)
        graphs.append((gr, side))
    for turn in range(3):
        for s in sides:
            s["start"] += 7 + turn
            s["lens"].copy_(s["start"] + n_new)
            s["k"].copy_(make(H_kv))
            s["q"].copy_(make(H_q))
            s["table"].copy_(s["table"].flip(1))
        torch.cuda.synchronize()
        for gr, side in graphs:
            with torch.cuda.stream(side):
                gr.replay()
        torch.cuda.synchronize()
        for s in sides:
            want, want_l = binding.paged_attn(s["q"], s["cache"], s["table"], s["lens"])
            assert torch.equal(s["out"], want) and torch.equal(s["lse"], want_l)


def test_on_another_stream():
    pool = Pool("e4m3", 2, 64, 64, [3000], 47, seed=12)
    q = torch.randn(1, 1, 8, 64, device=DEV).to(torch.bfloat16)
    want, want_l = binding.paged_attn(q, pool.cache, pool.table_d, ints([3000]))
    lens = ints([3000])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = binding.paged_attn(q, pool.cache, pool.table_d, lens, stream=side)
    k, v = binding.paged_read(pool.cache, pool.table_d, None, 3000, stream=side)
    binding.paged_append(pool.cache, pool.table_d, k, v, ints([0]), stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_l)


def test_pages_past_32_bit_offsets():
    """A pool of more than 2^32 values a tensor: its first and its last pages."""
    H, page, D = 8, 128, 128
    n = (1 << 32) // (H * page * D) + 40
    cache = binding.PagedCache(*(torch.empty(n, H, page, D, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)),
                               *(torch.empty(n, H, page, dtype=torch.uint8, device=DEV) for _ in range(2)))
    table = ints([[n - 1, 0, n - 7]])
    k, v = (torch.randn(1, 300, H, D, device=DEV).to(torch.bfloat16) for _ in range(2))
    st = status_word()
    binding.paged_append(cache, table, k, v, ints([0]), dev_status=st)
    back = binding.paged_read(cache, table, None, 300, dev_status=st)
    small = binding.paged_cache(3, H, page, D, dtype=E4M3)
    binding.paged_append(small, ints([[0, 1, 2]]), k, v, ints([0]), dev_status=st)
    for n_new in (1, 33):
        q = torch.randn(1, n_new, 2 * H, D, device=DEV).to(torch.bfloat16)
        got = binding.paged_attn(q, cache, table, ints([300]), dev_status=st)
        want = binding.paged_attn(q, small, ints([[0, 1, 2]]), ints([300]), dev_status=st)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    again = binding.paged_read(small, ints([[0, 1, 2]]), None, 300)
    assert torch.equal(back[0], again[0]) and torch.equal(back[1], again[1])
    assert int(st.item()) == 0


def test_malformed_offsets_and_lengths_stay_inside():
    """Offsets that fall, pass the rows or max_seqlen, lengths below 0 or past
    the table: nothing outside the tensors is read or written."""
    pool = Pool("bf16", 2, 16, 64, [64, 64], 4, seed=13)
    q = torch.randn(20, 4, 64, device=DEV).to(torch.bfloat16)
    for cu, lens, mx in (([0, 12, 3], [64, 64], 8), ([-5, 500, 600], [1 << 30, -9], 300), ([3, 9, 18], [64, 5], 2)):
        out = torch.full((20, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((4, 20), 7.0, device=DEV)
        binding.paged_attn_varlen(q, pool.cache, pool.table_d, ints(lens), ints(cu), mx, out=out, lse=lse)
        torch.cuda.synchronize()
        assert bool(out.isfinite().all())
    st = status_word()
    binding.paged_append_varlen(pool.cache, pool.table_d, q[:, :2].contiguous(), q[:, :2].contiguous(), ints([0, 12, 3]),
                                ints([1 << 30, -(1 << 30)]), dev_status=st)
    assert int(st.item()) == RANGE


def test_both_libraries_agree():
    """The bounds-checked build: the same bits, and no access out of range."""
    for kind in ("bf16", "e4m3"):
        pool = Pool(kind, 2, 16, 64, [501, 33, 0], 32, seed=14)
        k = torch.randn(3, 1, 2, 64, device=DEV).to(torch.bfloat16)
        res = {}
        for variant in ("release", "debug"):
            prev = binding.use_library(variant)
            try:
                st = status_word()
                got = []
                binding.paged_append(pool.cache, pool.table_d, k, k, ints([500, 32, 0]), n_new=ints([1, 1, 0]), dev_status=st)
                for n_new in (1, 3, 30):
                    q = torch.randn(3, n_new, 8, 64, generator=torch.Generator(device=DEV).manual_seed(n_new), device=DEV)
                    got += binding.paged_attn(q.to(torch.bfloat16), pool.cache, pool.table_d, ints([501, 33, 0]), dev_status=st)
                torch.cuda.synchronize()
                assert int(st.item()) == 0
                got += binding.paged_read(pool.cache, pool.table_d, ints([0, 30, 0]), 2, dev_status=st)
                torch.cuda.synchronize()
                assert int(st.item()) == RANGE              # the empty sequence's slots
                res[variant] = got
            finally:
                binding.use_library(prev)
        for x, y in zip(res["release"], res["debug"]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def reference(q, cache, table, lens, news, rows, window, n_sink):
    """(out, lse, terms) of sampled packed rows in float64 on the GPU; terms are
    the sums that the tolerances are made of: of |s|'s addends, of p |v|."""
    page, D = cache.dims[2], cache.dims[3]
    H_kv, H_q = cache.dims[1], q.shape[1]
    k, v = (t.double() if len(cache) == 2 else t.view(torch.uint8).view(E4M3).double() for t in cache[:2])
    if len(cache) > 2:
        k, v = (t * torch.exp2(e.double() - 127)[..., None] for t, e in zip((k, v), cache[2:]))
    first = np.concatenate([[0], np.cumsum(news)])
    res = []
    for r in rows:
        b = int(np.searchsorted(first, r, side="right") - 1)
        p = lens[b] - news[b] + (r - first[b])
        j = torch.arange(p + 1, device=DEV)
        if window:
            j = j[(j > p - window) | (j < n_sink)]
        at, row = table[b, j // page].long(), j % page
        kk, vv = (x[at, :, row].repeat_interleave(H_q // H_kv, 1) for x in (k, v))      # [n, H_q, D]
        x = q[r].double()
        s = (kk * x).sum(-1) * D ** -0.5                                                # [n, H_q]
        lse = torch.logsumexp(s, 0)
        w = torch.exp(s - lse)
        e = ((kk * x).abs().sum(-1) * D ** -0.5).amax(0) * (D + 8) * 2.0 ** -23
        rel = 2 * e + 2.0 ** -20 * (1 + s.abs().amax(0)) + j.numel() * 2.0 ** -24
        res.append(((w[..., None] * vv).sum(0), lse, rel, (w[..., None] * vv.abs()).sum(0)))
    return res


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", [
    # lens, new tokens, H_q, H_kv, D, page, window, n_sink, max_len: what the launch is cut by
    ([10000], [10000], 4, 4, 64, 64, 0, 0, None),                   # more blocks than multiprocessors, and a rest
    ([9000, 5000], [3000, 5000], 16, 4, 128, 16, 0, 0, None),       # packed, a rest
    ([9000, 5000], [3000, 5000], 8, 4, 128, 128, 700, 5, 1 << 20),  # head by head
    ([40000, 40000], [100, 100], 8, 1, 128, 128, 0, 0, None),       # a few blocks, cut many times
    ([70000, 50, 33000, 1], [1, 1, 1, 1], 8, 2, 64, 32, 0, 0, None),
    ([70000, 50, 33000, 2], [2, 2, 2, 2], 16, 2, 128, 16, 0, 0, None),
], ids=str)
def test_large_calls(case, kind):
    lens, news, H_q, H_kv, D, page, window, n_sink, max_len = case
    g = torch.Generator(device=DEV).manual_seed(sum(lens))
    width = -(-max(lens) // page)
    held = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(width, -(-(max_len or 0) // page))), -1, dtype=torch.int32, device=DEV)
    ids, at = torch.randperm(sum(held), generator=g, device=DEV).int(), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    cache = binding.paged_cache(sum(held), H_kv, page, D, dtype=torch.bfloat16 if kind == "bf16" else E4M3)
    n = max(lens)
    for lo in range(0, n, 8192):            # the whole axis, appended in pieces
        t = min(8192, n - lo)
        k, v = (torch.randn(len(lens), t, H_kv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        left = ints([min(max(x - lo, 0), t) for x in lens])
        binding.paged_append(cache, table, k, v, ints([lo] * len(lens)), n_new=left)
    q = torch.randn(sum(news), H_q, D, generator=g, device=DEV).to(torch.bfloat16)
    cu = ints(np.concatenate([[0], np.cumsum(news)]).tolist())
    st = status_word()
    out, lse = binding.paged_attn_varlen(q, cache, table, ints(lens), cu, max(news), max_len=max_len, window=window,
                                         n_sink=n_sink, dev_status=st)
    again, again_l = binding.paged_attn_varlen(q, cache, table, ints(lens), cu, max(news), max_len=max_len, window=window,
                                               n_sink=n_sink)
    assert int(st.item()) == 0
    assert torch.equal(out, again) and torch.equal(lse, again_l)
    ends = np.cumsum(news)
    rows = sorted(set(np.random.default_rng(0).integers(0, sum(news), 40).tolist()) | {0} | set((ends - 1).tolist()) |
                  {x for x in (127, 128, 255, 256, 5119) if x < sum(news)})
    u_w = 2.0 ** -8 if kind == "bf16" or max(news) * H_q // H_kv > 16 else 2.0 ** -11
    for r, (want, want_l, rel, pv) in zip(rows, reference(q, cache, table, lens, news, rows, window, n_sink)):
        assert bool(((out[r].double() - want).abs() <= want.abs() * 2.0 ** -8 + (rel + u_w)[:, None] * pv).all()), r
        assert bool(((lse[:, r].double() - want_l).abs() <= rel).all()), r


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,group,window", [(64, 1, 0), (128, 3, 0), (128, 4, 90), (64, 2, 200)])
def test_many_rows_keep_apart_too(kind, D, group, window):
    """Many rows: values that are not finite, in their tokens' own block and at
    the windows' edges, change no bit of the rows that do not see them, and
    reach their own dimensions of the rows that do."""
    lens, n_new, page, n_sink = 900, 330, 32, 5
    pool = Pool(kind, 1, page, D, [lens], 29, seed=22)
    q = torch.randn(1, n_new, group, D, device=DEV).to(torch.bfloat16)
    kw = dict(window=window, n_sink=n_sink)
    out, lse = binding.paged_attn(q, pool.cache, pool.table_d, ints([lens]), **kw)
    bad = [560, 575, 640, 703, 704, 899, 500, 433, 2]
    for j in bad:
        at, row = pool.table[0, j // page], j % page
        if kind == "bf16":
            pool.cache.v[at, 0, row, 1::5] = float("inf") if j % 2 else float("nan")
        else:
            pool.cache.v.view(torch.uint8)[at, 0, row, 1::5] = 0x7f
    got, got_l = binding.paged_attn(q, pool.cache, pool.table_d, ints([lens]), **kw)
    assert torch.equal(got_l, lse)
    for t in range(n_new):
        p = lens - n_new + t
        seen = any(j <= p and (window == 0 or j > p - window or j < n_sink) for j in bad)
        if seen:
            hit = torch.zeros(D, dtype=torch.bool, device=DEV)
            hit[1::5] = True
            assert not bool(got[0, t][:, hit].isfinite().any()), t
            assert torch.equal(got[0, t][:, ~hit], out[0, t][:, ~hit]), t
        else:
            assert torch.equal(got[0, t], out[0, t]), t


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_values_outside_the_block_may_be_anything(kind):
    """Many rows: values that no row of a block of tokens sees (the next
    block's, those behind every window, past the end) change no bit of its
    results, finite or not."""
    H, D, page = 1, 64, 16
    lens, n_new, group = 700, 400, 2                        # blocks of 128 tokens
    pool = Pool(kind, H, page, D, [lens], 50, seed=21)
    q = torch.randn(1, n_new, H * group, D, device=DEV).to(torch.bfloat16)
    kw = dict(window=150, n_sink=3)
    out, lse = binding.paged_attn(q, pool.cache, pool.table_d, ints([lens]), **kw)
    # the second block's tokens are at 428 to 555, the first sees 279 (151 + 128) to 427
    for slots in (range(428, lens), range(3, 300 - 150 + 1)):
        for j in slots:
            at, row = pool.table[0, j // page], j % page
            pool.cache.v.view(torch.uint8)[at, :, row] = 0x7f          # NaN in e4m3, in bf16 0x7f7f is finite
            if kind == "bf16":
                pool.cache.v[at, :, row] = float("nan")
    got, got_l = binding.paged_attn(q, pool.cache, pool.table_d, ints([lens]), **kw)
    assert torch.equal(got[:, :128], out[:, :128]) and torch.equal(got_l, lse)
    assert bool(got[:, 128:].isnan().all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_packed_calls_follow_each_other_without_waits(kind):
    """A packed call that may be long but is short (its offsets have fewer blocks than
    the launch makes whole ones, so that nothing is left to join), then the same slots
    written anew at once, offsets and lengths changing in place in between: each call
    sees what was there at its turn, as calls with waits between them do."""
    H, page, D, width, total = 16, 64, 64, 512, 4096
    g = torch.Generator(device=DEV).manual_seed(44)
    dtype = torch.bfloat16 if kind == "bf16" else E4M3
    q = torch.randn(total, H, D, generator=g, device=DEV).to(torch.bfloat16)
    news = [torch.randn(512, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(4)]
    steps = [([0, 300], 512), ([0, 30], 32768), ([0, 300], 32768), ([0, 4096], 9000), ([5, 6], 40), ([0, 300], 32768)]
    steps = [(ints(cu), ints([n])) for cu, n in steps]
    table = torch.randperm(width, generator=g, device=DEV).to(torch.int32)[None]
    full = torch.randn(1, width * page, H, D, generator=g, device=DEV).to(torch.bfloat16)

    def run(wait):
        cache = binding.paged_cache(width, H, page, D, dtype=dtype)
        binding.paged_append(cache, table, full, full, ints([0]))
        cu, lens, zero, rows = ints([0, 0]), ints([0]), ints([0]), ints([0, 512])
        res = []
        torch.cuda.synchronize()
        for i, (c, n) in enumerate(steps):
            cu.copy_(c)
            lens.copy_(n)
            binding.paged_append_varlen(cache, table, news[i % 4], news[(i + 1) % 4], rows, zero)
            if wait:
                torch.cuda.synchronize()
            out = torch.zeros_like(q)
            lse = torch.zeros(H, total, device=DEV)
            if wait:
                torch.cuda.synchronize()
            binding.paged_attn_varlen(q, cache, table, lens, cu, total, out=out, lse=lse)
            if wait:
                torch.cuda.synchronize()
            res += [out, lse]
        torch.cuda.synchronize()
        return res

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [[1] * 9, [40] * 9, [0] * 9, [1, 50] * 5 + [0] * 8], ids=["short", "long", "empty", "both"])
def test_short_sequences_have_their_own_launch(kind, news):
    """A bound on new tokens far above their mean: sequences of a few and of many rows
    are launched apart, and here one of the launches may find nothing. Pages that are not
    there are reported from both; rows of no sequence stay as they were."""
    H_q, H_kv, D, page, B, mx = 8, 2, 64, 16, len(news), 500
    lens = [max(n, 37 * (i + 1) % 300) for i, n in enumerate(news)]
    pool = Pool(kind, H_kv, page, D, lens, 2000, seed=46)
    g = torch.Generator().manual_seed(47)
    total = sum(news) + 5
    q = torch.randn(total, H_q, D, generator=g).to(torch.bfloat16)
    parts = [x.numpy() for x in torch.split(q[:-5].float(), news)]
    q = q.to(DEV)
    cu = np.concatenate([[0], np.cumsum(news)])
    n_bytes = binding.paged_attn_workspace_bytes(pool.cache, B, mx, H_q, 2000 * page, total=total)
    ws = torch.full((n_bytes,), 255, dtype=torch.uint8, device=DEV)      # NaN
    out, lse = torch.full_like(q, 7.0), torch.full((H_q, total), 7.0, device=DEV)
    st = status_word()
    binding.paged_attn_varlen(q, pool.cache, pool.table_d, ints(lens), ints(cu.tolist()), mx, out=out, lse=lse, workspace=ws,
                              dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool((out[cu[-1]:] == 7).all()) and bool((lse[:, cu[-1]:] == 7).all())
    k, v, has = pool.rows(max(lens))
    k, v = np.nan_to_num(k), np.nan_to_num(v)
    want, want_l = paged.attention(parts, k, v, lens, news, has, 0, 0)
    t_out, t_lse = bounds(parts, k, v, lens, news, has, 0, 0, want, 2.0 ** -8, D ** -0.5)
    for b, n in enumerate(news):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        check(out[rows], want[b], t_out[b], f"out of {b}")
        check(lse[:, rows], want_l[b], t_lse[b], f"lse of {b}")
    for gone in {int(np.argmax(news)), int(np.argmin([n if n else 1 << 20 for n in news]))}:
        if news[gone] == 0:
            continue
        table = pool.table_d.clone()
        table[gone, 0] = -1
        st = status_word()
        binding.paged_attn_varlen(q, pool.cache, table, ints(lens), ints(cu.tolist()), mx, workspace=ws, dev_status=st)
        assert int(st.item()) == RANGE
