"""How attention over pages is cut up, and what workspace that takes: host code alone."""

import ctypes

import pytest

from sequence_exact_attention_gb300 import binding

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
