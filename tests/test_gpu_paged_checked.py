"""The bounds-checked build over the paged cache's kernels: every table entry, page, part
and expanded tile that they reach lies inside its tensor, and the results are the
release build's, to the bit."""

import numpy as np
import pytest
import torch

from sequence_exact_attention_gb300 import binding

from test_gpu_paged import Pool, ints, status_word

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")

CASES = [
    # name, lens, new tokens, H_q, H_kv, D, page, width, window, n_sink
    ("few_rows_cut", [9000, 12, 4097], [2, 2, 2], 8, 1, 128, 16, 563, 0, 0),
    ("few_rows_window", [4000, 2100, 5], [3, 3, 3], 16, 4, 64, 64, 63, 300, 140),
    ("several_blocks", [515, 40, 129], [10, 4, 7], 8, 2, 128, 32, 33, 0, 0),
    ("pieces", [700, 0, 300, 257], [300, 0, 61, 200], 10, 2, 128, 16, 44, 0, 0),
    ("pieces_window", [3000, 2500], [700, 513], 8, 2, 64, 32, 100, 700, 5),
    ("pieces_cut", [9000, 7000], [60, 100], 8, 2, 128, 128, 71, 0, 0),
    ("short_beside_long", [900, 1, 64, 700, 0, 2, 33, 17, 500, 1], [1, 1, 4, 300, 0, 2, 1, 17, 5, 1], 8, 2, 128, 16, 2000, 0, 0),
    ("by_page", [700, 33, 0, 1500, 900, 64, 129, 400, 10, 2000], [300, 1, 0, 40, 2, 64, 3, 100, 1, 1], 16, 8, 128, 32, 4096, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_both_builds_agree(case, kind):
    _, lens, news, H_q, H_kv, D, page, width, window, n_sink = case
    pool = Pool(kind, H_kv, page, D, lens, width, seed=7)
    old = [t.view(torch.uint8).clone() for t in pool.cache]
    g = torch.Generator(device=DEV).manual_seed(8)
    total = sum(news)
    q, k, v = (torch.randn(total, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (H_q, H_kv, H_kv))
    cu = ints(np.concatenate([[0], np.cumsum(news)]).tolist())
    start = ints([n - m for n, m in zip(lens, news)])
    kw = dict(window=window, n_sink=n_sink)
    n_bytes = binding.paged_attn_workspace_bytes(pool.cache, len(lens), max(news), H_q, width * page, total=total, **kw)
    res = {}
    for variant in ("release", "debug"):
        prev = binding.use_library(variant)
        try:
            for t, x in zip(pool.cache, old):
                t.view(torch.uint8).copy_(x)
            st = status_word()
            binding.paged_append_varlen(pool.cache, pool.table_d, k, v, cu, start, dev_status=st)
            ws = torch.full((n_bytes,), 255, dtype=torch.uint8, device=DEV)
            out, lse = torch.zeros_like(q), torch.zeros(H_q, total, device=DEV)
            binding.paged_attn_varlen(q, pool.cache, pool.table_d, ints(lens), cu, max(news), out=out, lse=lse, workspace=ws,
                                      dev_status=st, **kw)
            torch.cuda.synchronize()
            assert int(st.item()) == 0
            got = [out, lse, *pool.cache]
            if len(set(news)) == 1:
                got += binding.paged_attn(q.view(len(lens), news[0], H_q, D), pool.cache, pool.table_d, ints(lens),
                                          dev_status=st, **kw)
                assert int(st.item()) == 0
            got += binding.paged_read(pool.cache, pool.table_d, start, max(news))
            res[variant] = [x.view(torch.uint8).clone() for x in got]
        finally:
            binding.use_library(prev)
    for x, y in zip(res["release"], res["debug"]):
        assert torch.equal(x, y)
