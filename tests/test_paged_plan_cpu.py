"""How attention over pages is cut up, and what workspace that takes: host code alone."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from sequence_exact_attention_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sequence_exact_attention_gb300", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
OK, RANGE = 0, 10


def workspace(lib, B, S_q, H_q, max_len, H, D, kind, total=None, window=0, n_sink=0, page=64):
    """(status, bytes) of a call of these sizes."""
    n = ctypes.c_size_t()
    pages = binding._pages((0,) * (4 if kind == "e4m3" else 2), (64, H, page, D), kind == "e4m3")
    st = lib.paged_attn_workspace(pages, B, S_q, total or 0, H_q, max_len, window, n_sink, total is not None,
                                  ctypes.byref(n))
    return st, n.value


@pytest.mark.parametrize("D,H", [(128, 64), (64, 128)])
def test_an_expansion_too_large_is_refused_before_anything_runs(lib, D, H):
    """8-bit pages and a piece of a prompt: what the kernel that expands the pages cannot
    count is out of range from the start, not after another launch of the same call."""
    size = dict(B=1, S_q=100, H_q=H, H=H, D=D, kind="e4m3")
    assert workspace(lib, max_len=1 << 30, **size)[0] == RANGE
    assert workspace(lib, max_len=(1 << 30) - 128, **size)[0] == OK


@pytest.mark.parametrize("B", [64, 256, 1000])
@pytest.mark.parametrize("T,total", [(512, 575), (512, None), (4096, 9000)])
@pytest.mark.parametrize("n_pages", [4096, 1 << 20])
def test_the_workspace_of_8_bit_pages_is_bounded(lib, B, T, total, n_pages):
    """It does not grow with the number of sequences, nor with a table that is wider than
    the pool is large; a long sequence's own tiles are always in it."""
    H, D, page, limit = 8, 128, 64, 4 << 30
    for max_len in (8192, 1 << 17, 1 << 20):
        n = ctypes.c_size_t()
        pages = binding._pages((0,) * 4, (n_pages, H, page, D), True)
        assert lib.paged_attn_workspace(pages, B, T, total or 0, 32, max_len, 0, 0, total is not None, ctypes.byref(n)) == OK
        tiles = -(-max_len // 128) * H * 128 * D * 4
        # and partial results: of at most eight waves of blocks, chunks of 256 rows
        parts = 9 * 152 * 256 * (D + 2) * 4
        assert n.value <= max(limit, tiles) + parts, (max_len, n.value)
        if n_pages * page <= limit // (H * D * 4):
            assert n.value <= limit + parts


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers are not available")
    out = str(tmp_path_factory.mktemp("paged") / "libpaged.so")
    cmd = [gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(CUDA, "include"), os.path.join(ROOT, "tests", "paged_harness.cpp"),
           os.path.join(CSRC, "paged_plan.cpp"), "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return ctypes.CDLL(out)


WALKS = [
    # lens, new tokens, H_q, H_kv, D, window, n_sink, max_len, pages of the pool, packed
    ([4096], [1], 32, 8, 128, 0, 0, 4096, 64, False),
    ([4096], [1], 32, 8, 128, 0, 0, 1 << 17, 64, False),
    ([8192, 1, 0, 77], [1] * 4, 8, 2, 64, 0, 0, 9000, 256, False),
    ([3, 5, 0], [5] * 3, 4, 4, 64, 0, 0, 48, 8, False),
    ([5000, 130, 700, 31], [4] * 4, 8, 2, 128, 300, 5, 6000, 256, False),
    ([5000, 4000], [6] * 2, 16, 2, 128, 1000, 200, 5000, 256, False),
    ([20000, 333], [1, 1], 40, 2, 64, 129, 4000, 20000, 512, False),
    ([2000, 1500, 900], [400] * 3, 8, 2, 64, 0, 0, 2000, 256, False),
    ([9000], [1000], 4, 2, 128, 700, 129, 9000, 256, False),
    ([100000], [64], 8, 8, 128, 0, 0, 100000, 2048, False),
    ([400, 300], [300] * 2, 5, 1, 64, 0, 0, 1 << 20, 32, False),
    ([3000, 100, 3000, 4096, 1290, 3223], [3000, 0, 1000, 1, 777, 222], 8, 2, 64, 0, 0, 4096, 256, True),
    ([3000, 100, 3000, 4096, 1290, 3223], [3000, 0, 1000, 1, 777, 222], 8, 2, 64, 600, 3, 1 << 17, 256, True),
    ([2048] * 9 + [4000] + [1] * 6, [1] * 9 + [512] + [1] * 5 + [0], 32, 8, 128, 0, 0, 8192, 1024, True),
    ([500] * 30 + [800], [1] * 30 + [300], 8, 8, 128, 0, 0, 1 << 17, 1024, True),
    ([500] * 30 + [800], [1] * 30 + [300], 8, 8, 128, 0, 0, 1 << 17, 1 << 18, True),
    ([500 + 10 * i for i in range(21)], [20 + 5 * i for i in range(21)], 8, 8, 128, 0, 0, 1 << 17, 1 << 18, True),
    ([500 + 10 * i for i in range(21)], [130] * 21, 8, 8, 128, 0, 0, 1 << 17, 1 << 18, False),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", WALKS, ids=str)
def test_every_visible_tile_is_in_one_chunk(harness, case, kind):
    """Every query row of every sequence and head has one block, whose CTAs walk each tile
    of slots that one of its rows sees once, and no other; chunks have parts of their own
    within the workspace, and what is expanded covers what is walked."""
    lens, news, H_q, H_kv, D, window, n_sink, max_len, n_pages, packed = case
    B, grp, total = len(lens), H_q // H_kv, sum(news)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    lens_c = np.array(lens, np.int32)
    rows, launches = np.zeros((1 << 20, 9), np.int32), np.zeros((64, 4), np.int32)
    ip = ctypes.POINTER(ctypes.c_int)
    ptr = lambda x: x.ctypes.data_as(ip)    # noqa: E731
    n = harness.ra_paged_walks(B, max(news), total, H_q, H_kv, D, 64, n_pages, int(kind == "e4m3"), max_len, window, n_sink,
                               ptr(lens_c), ptr(cu) if packed else None, ptr(rows), len(rows), ptr(launches), len(launches))
    assert 0 < n <= len(rows)
    eff = 0 if window >= max_len else window
    blocks, parts = {}, {}
    for launch, b, h, r0, R, tile, split, lo, part in rows[:n].tolist():
        blk = blocks.setdefault((b, h, r0), [launch, R, tile, [], set()])
        assert blk[:3] == [launch, R, tile], "one launch has the block"
        if lo >= 0:
            blk[3].append(lo)
        if part >= 0:
            blk[4].add(split)
            assert part + launches[launch, 0] <= launches[launch, 1]
            assert parts.setdefault((launch, part), (b, h, r0, split)) == (b, h, r0, split)
        else:
            assert split == -1
    for b in range(B):
        for h in range(H_kv):
            mine = sorted(x for x in blocks if x[:2] == (b, h))
            covered = [r for x in mine for r in range(x[2], x[2] + blocks[x][1])]
            assert covered == list(range(news[b] * grp)), (b, h)
            for x in mine:
                launch, R, tile, got, _ = blocks[x]
                j = np.arange(max(lens[b], 1))
                p = lens[b] - news[b] + np.unique((x[2] + np.arange(R)) // grp)[:, None]
                see = (j <= p) & ((eff == 0) | (j > p - eff) | (j < n_sink))
                want = np.unique(j[see.any(0)] // tile * tile).tolist()
                assert sorted(got) == want, x
                if kind == "e4m3" and launches[launch, 0] > 16 and launches[launch, 3] >= 0:
                    assert len(want) <= launches[launch, 3]
