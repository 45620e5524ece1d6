"""Pieces of prompts over 8-bit pages where the table is far wider than the sequences are
long: what is expanded stays bounded (page by page of a small pool, some sequences at a
time of a large one), and the results are those of any other call. Tolerances as in
tests/test_gpu_paged.py, those of weights that are rounded to bf16 (2^-8)."""

import numpy as np
import pytest
import torch

from oracle import paged
from sequence_exact_attention_gb300 import binding

from test_gpu_paged import E4M3, RANGE, Pool, bounds, check, ints, status_word

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
WIDE = 1 << 17                  # slots of a table's row

CASES = [
    # name, lens, new tokens, H_q, H_kv, D, page, window, n_sink, a large pool
    ("by_page", [700, 33, 0, 1500, 900, 64, 129, 400, 10, 2000], [300, 1, 0, 40, 2, 64, 3, 100, 1, 1], 16, 8, 128, 32, 0, 0,
     False),
    ("by_page_window", [17000, 16500] + [20 + i for i in range(68)], [40, 27] + [1 + i % 3 for i in range(68)], 16, 8, 128, 16,
     16000, 5, False),
    ("by_page_padded", [300 + 50 * i for i in range(9)], [60] * 9, 8, 8, 128, 64, 0, 0, False),
    ("groups", [700, 33, 0, 1500, 900, 64, 129, 400, 10, 2000], [300, 1, 0, 40, 2, 64, 3, 100, 1, 1], 16, 8, 128, 32, 0, 0,
     True),
    ("groups_all_long", [700, 330, 100, 1500, 900, 164, 129, 400, 110], [300, 130, 100, 340, 122, 64, 31, 100, 10], 8, 8, 128,
     64, 0, 0, True),
    ("groups_window", [120 + i for i in range(69)] + [17000], [25 + i % 5 for i in range(68)] + [0, 30], 16, 8, 128, 64, 16000,
     130, True),
    ("groups_padded", [300 + 50 * i for i in range(9)], [60] * 9, 16, 8, 128, 64, 0, 0, True),
    ("groups_of_d64", [300 + 50 * i for i in range(19)], [49] * 19, 8, 8, 64, 128, 0, 0, True),
]


def spread(pool, n, seed):
    """The pool's pages in a pool of n, among pages of NaN, and their table."""
    _, H, page, D = pool.shape
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:pool.n]
    parts = []
    for t in pool.cache:
        big = torch.full((n, *t.shape[1:]), 127, dtype=torch.uint8, device=DEV)
        big[ids.to(DEV)] = t.view(torch.uint8)
        parts.append(big.view(t.dtype))
    table = np.where(pool.table >= 0, ids.numpy()[pool.table], -1).astype(np.int32)
    return binding.PagedCache(*parts), torch.from_numpy(table).to(DEV)


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_a_table_far_wider_than_the_sequences(case):
    _, lens, news, H_q, H_kv, D, page, window, n_sink, large = case
    pool = Pool("e4m3", H_kv, page, D, lens, WIDE // page, seed=sum(lens))
    n_pages = (1 << 30) // (H_kv * page * D) + 5 if large else pool.n + 2
    cache, table = spread(pool, n_pages, len(lens))
    g = torch.Generator().manual_seed(5)
    q = torch.randn(sum(news), H_q, D, generator=g).to(torch.bfloat16)
    parts = [x.numpy() for x in torch.split(q.float(), news)]
    want, want_l, t_out, t_lse = [], [], [], []
    for b, (x, n, new) in enumerate(zip(parts, lens, news)):         # (one at a time: they differ in length)
        k, v = (np.nan_to_num(paged.rows(y, pool.table[b:b + 1], n)) for y in pool.values)
        has = np.ones((1, n), bool)
        o, l = paged.attention([x], k, v, [n], [new], has, window, n_sink)
        t, u = bounds([x], k, v, [n], [new], has, window, n_sink, o, 2.0 ** -8, D ** -0.5)
        for y, z in zip((want, want_l, t_out, t_lse), (o, l, t, u)):
            y += z
    cu = np.concatenate([[0], np.cumsum(news)])
    qp = torch.cat([q, torch.full((3, H_q, D), float("nan"), dtype=q.dtype)]).to(DEV)
    out, lse = torch.full_like(qp, 7.0), torch.full((H_q, sum(news) + 3), 7.0, device=DEV)
    st = status_word()
    n_bytes = binding.paged_attn_workspace_bytes(cache, len(lens), max(news), H_q, WIDE, window, n_sink, total=sum(news) + 3)
    assert n_bytes < (5 << 30)
    ws = torch.full((n_bytes + 64,), 255, dtype=torch.uint8, device=DEV)          # NaN
    binding.paged_attn_varlen(qp, cache, table, ints(lens), ints(cu.tolist()), max(news), window=window, n_sink=n_sink,
                              out=out, lse=lse, workspace=ws[:n_bytes], dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool((ws[n_bytes:] == 255).all())
    assert bool((out[-3:] == 7).all()) and bool((lse[:, -3:] == 7).all())
    for b in range(len(lens)):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        check(out[rows], want[b], t_out[b], f"out of {b}")
        check(lse[:, rows], want_l[b], t_lse[b], f"lse of {b}")
    # again, over what the first call left behind
    again, again_l = binding.paged_attn_varlen(qp, cache, table, ints(lens), ints(cu.tolist()), max(news), window=window,
                                               n_sink=n_sink, workspace=ws)
    assert torch.equal(again[:-3], out[:-3]) and torch.equal(again_l[:, :-3], lse[:, :-3])
    if len(set(news)) == 1:
        B, T = len(news), news[0]
        out1, lse1 = binding.paged_attn(q.view(B, T, H_q, D).to(DEV), cache, table, ints(lens), window=window, n_sink=n_sink,
                                        workspace=ws, dev_status=st)
        assert int(st.item()) == 0
        for b in range(B):
            check(out1[b], want[b], t_out[b], f"padded out of {b}")
            check(lse1[b], want_l[b], t_lse[b], f"padded lse of {b}")
    # a page that is not there
    b = int(np.argmax(news))
    table[b, 0] = -1
    binding.paged_attn_varlen(qp, cache, table, ints(lens), ints(cu.tolist()), max(news), dev_status=st)
    assert int(st.item()) == RANGE


@pytest.mark.parametrize("large", [False, True])
def test_a_captured_step_over_a_wide_table(large):
    """Its lengths, offsets and pages change between replays."""
    H_q, H, D, page, B, T = 8, 8, 128, 64, 10, 96
    pool = Pool("e4m3", H, page, D, [900] * B, WIDE // page, seed=3)
    cache, table = spread(pool, (1 << 30) // (H * page * D) + 5 if large else pool.n, 1)
    g = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn(B * T, H_q, D, generator=g, device=DEV).to(torch.bfloat16)
    lens, cu = ints([900] * B), ints([0] * (B + 1))
    out, lse = torch.zeros_like(q), torch.zeros(H_q, B * T, device=DEV)
    ws = torch.empty(binding.paged_attn_workspace_bytes(cache, B, T, H_q, WIDE, total=B * T), dtype=torch.uint8, device=DEV)

    def step():
        binding.paged_attn_varlen(q, cache, table, lens, cu, T, out=out, lse=lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for news in ([T] * B, [1] * B, [0, 96, 5, 0, 40, 17, 1, 1, 96, 0], [0] * B):
        lens.copy_(ints([900 - 31 * i - news[i] for i in range(B)]))
        cu.copy_(ints(np.concatenate([[0], np.cumsum(news)]).tolist()))
        table.copy_(table.flip(0))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got, got_l = out.clone(), lse.clone()
        out.fill_(7.0)
        lse.fill_(7.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(lse, got_l)
        assert bool((got[sum(news):] == 7).all())
        assert bool(got[:sum(news)].isfinite().all())
