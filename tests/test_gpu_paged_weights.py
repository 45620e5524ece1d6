"""Attention over the paged cache: softmax weights as exact as each kernel says.

    bf16 pages, up to 16 query rows a key/value head     2^-16 of a weight (two bf16 numbers)
    8-bit pages, up to 48 rows                           2^-11 (halves), or 2^-25 of the row's largest
    more rows                                            2^-8 (bf16)

and over 8-bit pages the second also for the short sequences of a packed call with
longer ones, where its bounds are wide. The other terms are those of
tests/test_gpu_paged.py. The outputs' own rounding, 2^-8 of them, would hide a weight's,
so here outputs cancel as well: half the slots have the weight 1 and the value x, the others a
weight just above 1, by less than a bf16 number's half step, and the value -x.
"""

import numpy as np
import pytest
import torch

from oracle import paged
from sequence_exact_attention_gb300 import binding

from test_gpu_paged import CASES, Pool, bounds, check, ints, status_word
from test_gpu_paged_range import far_bound, filled, held

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


def claimed(kind, rows):
    """A weight's relative error in a call of so many rows a head."""
    if kind == "bf16":
        return 2.0 ** -16 if rows <= 16 else 2.0 ** -8
    return 2.0 ** -11 if rows <= 48 else 2.0 ** -8


def cancelling(n, H, D, T, H_q, seed=0):
    """k, v [n, H, D] and q [T, H_q, D] whose outputs cancel."""
    g = torch.Generator().manual_seed(seed)
    k, v = torch.zeros(n, H, D), torch.randn(n // 2, 1, D, generator=g).repeat_interleave(2, 0).expand(n, H, D).clone()
    k[1::2, :, 0] = 0.9 * 2.0 ** -8 * D ** 0.5          # a logit of 0.9 2^-8 for queries of 1
    v[1::2] *= -1
    q = torch.zeros(T, H_q, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    return k, v, q


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,group", [(1, 1), (1, 8), (4, 4), (1, 16), (5, 5), (6, 8), (1, 20)])
@pytest.mark.parametrize("D", [64, 128])
def test_outputs_that_cancel(kind, T, group, D):
    n, H = 200, 2
    k, v, q = cancelling(n, H, D, T, H * group)
    cache, table = filled(kind, k, v)
    st = status_word()
    out, lse = binding.paged_attn(q[None].to(DEV), cache, table, ints([n]), dev_status=st)
    assert int(st.item()) == 0
    kk, vv = held(cache, table, n)
    x, has = [q.double().numpy()], np.ones((1, n), bool)
    want, want_l = paged.attention(x, kk, vv, [n], [T], has)
    u_w = claimed(kind, T * group)
    t_out, t_lse = bounds(x, kk, vv, [n], [T], has, 0, 0, want, u_w, D ** -0.5)
    if u_w == 2.0 ** -11:
        t_out[0] += far_bound(x[0], kk, vv, n, D ** -0.5)
    check(out[0], want[0], t_out[0], "out")
    check(lse[0], want_l[0], t_lse[0], "lse")


def test_short_sequences_beside_a_long_one_cancel():
    """8-bit pages, one new token a sequence and one piece of 100, tables far wider: the
    single tokens' weights are halves, whatever the piece's are."""
    n, H, D, group, B, page = 200, 2, 128, 4, 20, 32
    k, v, q = cancelling(n, H, D, B - 1 + 100, H * group)
    cache, table = filled("e4m3", k, v, page)
    wide = torch.full((B, 2000), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    cu = ints([0] + list(range(1, B)) + [B - 1 + 100])
    out, _ = binding.paged_attn_varlen(q.to(DEV), cache, wide, ints([n] * B), cu, 100)
    kk, vv = held(cache, table, n)
    x, has = [q[:1].double().numpy()], np.ones((1, n), bool)
    want, _ = paged.attention(x, kk, vv, [n], [1], has)
    t_out, _ = bounds(x, kk, vv, [n], [1], has, 0, 0, want, 2.0 ** -11, D ** -0.5)
    t_out[0] += far_bound(x[0], kk, vv, n, D ** -0.5)
    for b in range(B - 1):
        check(out[b:b + 1], want[0], t_out[0], f"out of {b}")


# (those of up to 16 or 48 rows a head; the others are held to 2^-8 already)
EXACT = [(c, kind) for c in CASES for kind in ("bf16", "e4m3") if claimed(kind, max(c[2]) * c[3] // c[4]) < 2.0 ** -8]


@pytest.mark.parametrize("case,kind", EXACT, ids=[f"{c[0]}-{kind}" for c, kind in EXACT])
def test_random_values(case, kind):
    """The cases of tests/test_gpu_paged.py whose sequences' rows all go one way."""
    _, lens, news, H_q, H_kv, D, page, width, window, n_sink = case
    u_w = claimed(kind, max(news) * H_q // H_kv)
    pool = Pool(kind, H_kv, page, D, lens, width, seed=sum(lens) + D)
    q = torch.randn(sum(news), H_q, D, generator=torch.Generator().manual_seed(15)).to(torch.bfloat16)
    parts = [x.numpy() for x in torch.split(q.float(), news)]
    k, v, has = pool.rows(max(max(lens), 1))
    k, v = np.nan_to_num(k), np.nan_to_num(v)
    want, want_l = paged.attention(parts, k, v, lens, news, has, window, n_sink)
    t_out, t_lse = bounds(parts, k, v, lens, news, has, window, n_sink, want, u_w, D ** -0.5)
    cu = np.concatenate([[0], np.cumsum(news)])
    out, lse = binding.paged_attn_varlen(q.to(DEV), pool.cache, pool.table_d, ints(lens), ints(cu.tolist()), max(news),
                                         window=window, n_sink=n_sink)
    for b in range(len(news)):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        # (2^-25 of the largest weight a slot is within the bound's n 2^-24 for sums of n terms)
        check(out[rows], want[b], t_out[b], f"out of {b}")
        check(lse[:, rows], want_l[b], t_lse[b], f"lse of {b}")
