"""Attention over the paged cache where numbers of one call lie far apart: a value, a
query or a score many powers of two above the others costs those no precision, in any
dimension, whichever kernel the call's size selects, and an infinity keeps its sign.

Tolerances are those of tests/test_gpu_paged.py, dimension by dimension: (relative
error of a weight) times the sum of w |v| of that dimension alone, plus 2^-8 of the
output. Over 8-bit pages, up to 48 rows a key/value head, a weight is a half: off by
2^-11 of itself, or, far below the row's largest weight, by 2^-25 of that one (half of
half's least step, where the weight 1 is 1).
"""

import numpy as np
import pytest
import torch

from oracle import paged
from sequence_exact_attention_gb300 import binding

from test_gpu_paged import E4M3, bounds, check, ints, status_word

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
INF = float("inf")


def held(cache, table, n):
    """Keys and values [1, H, n, D] float64 that the pages hold for the first n slots."""
    if len(cache) == 2:
        pools = [t.double().cpu().numpy() for t in cache]
    else:
        pools = [paged.values(t.view(torch.uint8).cpu().numpy(), e.cpu().numpy()) for t, e in zip(cache[:2], cache[2:])]
    return [paged.rows(x, table.cpu().numpy(), n) for x in pools]


def filled(kind, k, v, page=32, seed=0):
    """A cache that holds k, v [n, H, D], its pages in no order, and its table."""
    n, H, D = k.shape
    width = -(-n // page)
    g = torch.Generator(device=DEV).manual_seed(seed)
    table = torch.randperm(width + 2, generator=g, device=DEV).int()[None, :width].contiguous()
    cache = binding.paged_cache(width + 2, H, page, D, dtype=torch.bfloat16 if kind == "bf16" else E4M3)
    k, v = (x[None].to(DEV) for x in (k, v))
    binding.paged_append(cache, table, k, v, ints([0]))
    return cache, table


def far_bound(q, k, v, n, scale):
    """2^-25 of each row's largest weight, times every visible slot's |v|."""
    T, H_q, D = q.shape
    grp = H_q // k.shape[1]
    t = np.zeros(q.shape)
    for i in range(T):
        for h in range(H_q):
            seen = n - T + i + 1
            s = scale * (k[0, h // grp, :seen] @ q[i, h])
            w = np.exp(s - s.max())
            t[i, h] = 2.0 ** -25 / w.sum() * np.abs(v[0, h // grp, :seen]).sum(0)
    return t


def compare(kind, cache, table, q, n):
    """Runs q [T, H_q, D] as the last tokens of n slots and compares each dimension."""
    T, H_q, D = q.shape
    st = status_word()
    out, lse = binding.paged_attn(q[None].to(DEV), cache, table, ints([n]), dev_status=st)
    assert int(st.item()) == 0
    k, v = held(cache, table, n)
    x = [q.double().numpy()]
    has = np.ones((1, n), bool)
    want, want_l = paged.attention(x, k, v, [n], [T], has)
    halves = kind == "e4m3" and T * H_q // k.shape[1] <= 48
    u_w = 2.0 ** -11 if halves else 2.0 ** -8
    t_out, t_lse = bounds(x, k, v, [n], [T], has, 0, 0, want, u_w, D ** -0.5)
    if halves:
        t_out[0] += far_bound(x[0], k, v, n, D ** -0.5)
    check(out[0], want[0], t_out[0], "out")
    check(lse[0], want_l[0], t_lse[0], "lse")


ROWS = [(1, 1), (1, 4), (3, 4), (4, 8), (12, 4), (40, 4)]       # new tokens, group


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,group", ROWS)
@pytest.mark.parametrize("power", [10, 20, 30, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_one_far_larger_value(kind, T, group, power, D):
    """One value of one slot is 2^power, the others of its row are 0: every other
    dimension's outputs come from the other slots alone."""
    n, H = 333, 2
    g = torch.Generator().manual_seed(power + T)
    k, v = (torch.randn(n, H, D, generator=g) for _ in range(2))
    for at in (7, 200):
        v[at] = 0.0
        v[at, :, 3] = 2.0 ** power
    q = torch.randn(T, H * group, D, generator=g).to(torch.bfloat16)
    cache, table = filled(kind, k, v, seed=power)
    compare(kind, cache, table, q, n)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,group", [(1, 4), (4, 8), (40, 1)])
@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("outlier", [2.0 ** 10, 2.0 ** 16])
def test_a_leading_slot_with_a_far_larger_value(kind, T, group, late, outlier):
    """One slot has 2^14 times the others' weight, and a value far above theirs: together
    they weigh as much, and theirs are the other dimensions."""
    n, H, D = 16500, 1, 64
    g = torch.Generator().manual_seed(3)
    k, v = torch.zeros(n, H, D), torch.randn(n, H, D, generator=g) + 1.0
    at = n - T - 3 if late else 0
    k[at, :, 0] = 9.75                            # 8 * 9.75 / 8 nats, 2^14
    v[at] = 0.0
    v[at, :, 5] = outlier
    q = torch.zeros(T, H * group, D, dtype=torch.bfloat16)
    q[..., 0] = 8.0
    cache, table = filled(kind, k, v)
    compare(kind, cache, table, q, n)


@pytest.mark.parametrize("T,group", [(4, 2), (12, 4)])
@pytest.mark.parametrize("hidden", ["later", "window", "past"])
def test_a_hidden_scale_changes_nothing(T, group, hidden):
    """A slot's scale of 2^100 is nothing to the rows that do not see the slot, to the
    bit, in the same tile and in the same block of rows as one that does."""
    n, H, D = 170, 1, 128
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(n, H, D, generator=g) for _ in range(2))
    q = torch.randn(1, T, H * group, D, generator=g).to(torch.bfloat16).to(DEV)
    cache, table = filled("e4m3", k, v)
    n_seen = n if hidden != "past" else n - 5
    kw = dict(window=40, n_sink=1) if hidden == "window" else {}
    out, lse = binding.paged_attn(q, cache, table, ints([n_seen]), **kw)
    # "later": the last but one new token's; "window": what the second token has left behind
    at = {"later": n - 2, "window": n - T - 40 + 1, "past": n - 2}[hidden]
    page, row = int(table[0, at // 32]), at % 32
    cache.v_scale[page, :, row] = 227
    got, got_l = binding.paged_attn(q, cache, table, ints([n_seen]), **kw)
    assert torch.equal(got_l, lse)
    unseen = {"later": slice(0, T - 2), "window": slice(1, T), "past": slice(0, T)}[hidden]
    assert torch.equal(got[:, unseen], out[:, unseen])
    if hidden != "past":
        seen = T - 1 if hidden == "later" else 0
        assert float(got[0, seen].abs().max()) > 2.0 ** 80


@pytest.mark.parametrize("T,group", [(1, 4), (4, 2), (12, 4), (40, 4)])
@pytest.mark.parametrize("where", ["first", "last"])
def test_not_a_number_beside_a_far_larger_value(T, group, where):
    """A value that is not a number, in the same 16 slots as one of 2^40: its dimension of
    the rows that see it, and nothing else."""
    n, H, D = 250, 1, 128
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(n, H, D, generator=g) for _ in range(2))
    at = 33 if where == "first" else n - 1
    v[(at - 32) // 16 * 16 + 33] = 0.0
    v[(at - 32) // 16 * 16 + 33, :, 3] = 2.0 ** 40
    q = torch.randn(1, T, H * group, D, generator=g).to(torch.bfloat16).to(DEV)
    cache, table = filled("e4m3", k, v)
    out, lse = binding.paged_attn(q, cache, table, ints([n]))
    cache.v.view(torch.uint8)[int(table[0, at // 32]), :, at % 32, 9] = 0x7f
    got, got_l = binding.paged_attn(q, cache, table, ints([n]))
    assert torch.equal(got_l, lse)
    seen = T if where == "first" else 1
    assert bool(got[:, T - seen:, :, 9].isnan().all())
    got[:, T - seen:, :, 9] = out[:, T - seen:, :, 9]
    assert torch.equal(got, out)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,group", ROWS)
@pytest.mark.parametrize("power", [20, 40, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_one_far_larger_query_value(kind, T, group, power, D):
    """A query's one value of 2^power meets keys that are 0 there: the scores come from
    the others, those of the rows beside it as before, to the bit."""
    n, H = 300, 2
    g = torch.Generator().manual_seed(power + T)
    k, v = (torch.randn(n, H, D, generator=g) for _ in range(2))
    k[..., 5] = 0.0
    q = torch.randn(T, H * group, D, generator=g).to(torch.bfloat16)
    cache, table = filled(kind, k, v)
    before, before_l = binding.paged_attn(q[None].to(DEV), cache, table, ints([n]))
    q[::2, ::3, 5] = 2.0 ** power
    compare(kind, cache, table, q, n)
    after, after_l = binding.paged_attn(q[None].to(DEV), cache, table, ints([n]))
    same = torch.ones(T, H * group, dtype=torch.bool)
    same[::2, ::3] = False
    assert torch.equal(after[0][same], before[0][same])
    assert torch.equal(after_l[0].T[same], before_l[0].T[same])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,group", [(1, 1), (4, 2), (12, 1), (40, 4), (300, 1)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (120, 3)])
def test_infinite_values_keep_their_sign(D, T, group, window, n_sink):
    """bf16 pages: a value of infinity makes its dimension of the rows that see it infinite
    with its sign, and both signs, or a NaN, make it NaN: in whole tiles of slots, at a
    window's edges and among the new tokens, in calls of any size."""
    n = 700
    g = torch.Generator().manual_seed(T)
    k, v = (torch.randn(n, 1, D, generator=g) for _ in range(2))
    kw = dict(window=window, n_sink=n_sink)
    q = torch.randn(1, T, group, D, generator=g).to(torch.bfloat16).to(DEV)
    cache, table = filled("bf16", k, v)
    out, lse = binding.paged_attn(q, cache, table, ints([n]), **kw)
    bad = [(at, d, x) for at in (1, 100, 300, 450, n - T - 60, n - T, n - 2, n - 1)
           for d, x in ((at % 7, INF), (7 + at % 5, -INF), (12 + at % 3, float("nan")))]
    bad += [(20, 20, INF), (640, 20, INF), (640, 21, -INF), (1, 21, -INF), (699, 22, INF), (0, 22, -INF), (650, 23, -INF),
            (649, 23, INF)]
    for at, d, x in bad:
        cache.v[int(table[0, at // 32]), 0, at % 32, d] = x
    got, got_l = binding.paged_attn(q, cache, table, ints([n]), **kw)
    assert torch.equal(got_l, lse)
    want = out.clone()
    for t in range(T):
        p = n - T + t
        for at, d, x in bad:
            if at <= p and (window == 0 or at > p - window or at < n_sink):
                y = want[0, t, 0, d].item()
                want[0, t, :, d] = x if np.isfinite(y) else y + x
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], want[~nan])
