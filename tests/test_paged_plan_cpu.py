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
