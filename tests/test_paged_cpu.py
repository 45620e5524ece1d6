"""Refusals of the paged cache's entry points, before anything reaches a GPU."""

import copy
import ctypes

import pytest
import torch

from sequence_exact_attention_gb300 import binding

OK, NULL, SHAPE, HEADDIM, ALIGN, DTYPE, DEVICE, BUFFER, RANGE = 0, 1, 2, 3, 4, 5, 6, 9, 10
A = 0x10000000          # a 16-byte aligned fake address, never dereferenced
vp = ctypes.c_void_p


def addr(i, off=0):     # apart by more than any tensor below
    return vp(A + (i << 36) + off) if i else vp(0)


def pages(k=1, v=2, ks=0, vs=0, n=64, H=2, page=16, D=64, dtype=0, off=0):
    p = [a.value or 0 for a in (addr(k, off), addr(v), addr(ks), addr(vs))]
    return binding._PAGES.pack(*p, n, H, page, D, dtype)


def append(lib, table=5, width=8, k=6, v=7, start=8, n_new=0, B=2, T=3, dtype=0, off=0, p=None, **kw):
    pg = pages(**kw) if p is None else p
    return lib.paged_append(pg, addr(table), width, addr(k, off), addr(v), addr(start),
                            addr(n_new), B, T, dtype, None, None)


def test_append_refusals(lib):
    for bad in (dict(k=0), dict(v=0), dict(start=0), dict(table=0), dict(p=pages(k=0)), dict(p=pages(v=0)),
                dict(p=pages(dtype=2)), dict(p=pages(dtype=2, ks=9))):
        assert append(lib, **bad) == NULL, bad
    assert lib.paged_append(None, addr(5), 8, addr(6), addr(7), addr(8), None, 2, 3, 0, None, None) == NULL
    for bad in (dict(B=0), dict(T=0), dict(T=-1), dict(width=0), dict(n=0), dict(H=0), dict(page=8), dict(page=48),
                dict(page=256), dict(page=0)):
        assert append(lib, **bad) == SHAPE, bad
    assert append(lib, D=96) == HEADDIM
    assert append(lib, off=8) == ALIGN and append(lib, p=pages(off=8)) == ALIGN
    assert append(lib, dtype=2) == DTYPE and append(lib, p=pages(dtype=1)) == DTYPE
    assert append(lib, B=1 << 16, T=1 << 12, H=8, D=128) == RANGE
    assert append(lib, n=1 << 30, H=8) == RANGE
    assert append(lib, k=1) == BUFFER and append(lib, p=pages(v=1)) == BUFFER and append(lib, table=2) == BUFFER


def append_packed(lib, cu=8, n_seq=2, total=5, dtype=0):
    pg = pages()
    return lib.paged_append_varlen(pg, addr(5), 8, addr(6), addr(7), addr(9), addr(cu), n_seq, total,
                                   dtype, None, None)


def test_packed_append_refusals(lib):
    assert append_packed(lib, cu=0) == NULL
    assert append_packed(lib, n_seq=0) == SHAPE and append_packed(lib, total=0) == SHAPE
    assert append_packed(lib, dtype=3) == DTYPE
    assert append_packed(lib, cu=1) == BUFFER


def read(lib, k=6, v=7, T=3, dtype=0, **kw):
    pg = pages(**kw)
    return lib.paged_read(pg, addr(5), 8, None, addr(k), addr(v), 2, T, dtype, None, None)


def test_read_refusals(lib):
    assert read(lib, k=0, v=0) == NULL
    assert read(lib, T=0) == SHAPE and read(lib, page=12) == SHAPE
    assert read(lib, D=32) == HEADDIM and read(lib, dtype=2) == DTYPE
    assert read(lib, v=6) == BUFFER and read(lib, k=2) == BUFFER


def need(lib, B=2, S_q=1, total=0, H_q=4, max_len=128, window=0, n_sink=0, varlen=0, **kw):
    n, pg = ctypes.c_size_t(), pages(**kw)
    st = lib.paged_attn_workspace(pg, B, S_q, total, H_q, max_len, window, n_sink, varlen,
                                  ctypes.byref(n))
    return st, n.value


def attn(lib, q=6, table=5, width=8, lens=7, out=8, lse=9, B=2, S_q=1, H_q=4, max_len=128, window=0, n_sink=0, dtype=0,
         ws=10, ws_bytes=1 << 34, off=0, **kw):
    pg = pages(**kw)
    return lib.paged_attn(addr(q, off), pg, addr(table), width, addr(lens), addr(out), addr(lse), B,
                          S_q, H_q, max_len, window, n_sink, 0.0, dtype, addr(ws), ws_bytes, None, None)


def attn_packed(lib, cu=11, n_seq=2, total=7, max_seqlen=4, **kw):
    pg = pages(**kw)
    return lib.paged_attn_varlen(addr(6), pg, addr(5), 8, addr(7), addr(cu), addr(8), addr(9), n_seq,
                                 total, max_seqlen, 4, 128, 0, 0, 0.0, 0, addr(10), 1 << 34, None, None)


def test_attention_refusals(lib):
    for bad in (dict(q=0), dict(lens=0), dict(out=0), dict(table=0), dict(k=0)):
        assert attn(lib, **bad) == NULL, bad
    for bad in (dict(B=0), dict(S_q=0), dict(H_q=3), dict(H_q=0), dict(H_q=2 * 129), dict(H=0), dict(width=0)):
        assert attn(lib, **bad) == SHAPE, bad
    assert attn(lib, D=256) == HEADDIM
    assert attn(lib, dtype=1) == DTYPE and attn(lib, dtype=2) == DTYPE
    assert attn(lib, off=4) == ALIGN
    for bad in (dict(max_len=0), dict(max_len=129), dict(window=-1), dict(n_sink=-1), dict(width=1 << 27, max_len=(1 << 30) + 1),
                dict(B=1 << 15, S_q=1 << 10, H_q=16, H=16, D=128)):
        assert attn(lib, **bad) == RANGE, bad
    assert attn(lib, out=6) == BUFFER and attn(lib, out=1) == BUFFER and attn(lib, lse=7) == BUFFER
    long = dict(width=4096, max_len=65536)
    st, n = need(lib, max_len=65536)
    assert st == OK and n > 0
    assert attn(lib, ws_bytes=n - 1, **long) == BUFFER
    assert attn(lib, ws=0, **long) == NULL
    assert attn(lib, ws=6, **long) == BUFFER
    assert attn_packed(lib, cu=0) == NULL
    for bad in (dict(n_seq=0), dict(total=0), dict(max_seqlen=0)):
        assert attn_packed(lib, **bad) == SHAPE, bad


def test_workspace_refusals(lib):
    pg = pages()
    assert lib.paged_attn_workspace(pg, 2, 1, 0, 4, 128, 0, 0, 0, None) == NULL
    assert need(lib, page=24)[0] == SHAPE and need(lib, max_len=0)[0] == RANGE
    assert need(lib, varlen=1, total=0)[0] == SHAPE
    assert need(lib, B=1, S_q=1 << 24, H_q=128, H=1)[0] == RANGE


def test_the_binding_checks_tensors():
    with pytest.raises(ValueError, match="bfloat16 or float8"):
        binding.PagedCache(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64))
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    s = torch.zeros(2, 1, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="belong to"):
        binding.PagedCache(k, k.clone(), s, s.clone())
    with pytest.raises(ValueError, match="belong to"):
        binding.PagedCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="shape"):
        binding.PagedCache(k, k[:1])
    with pytest.raises(ValueError, match="contiguous"):
        binding.PagedCache(k.transpose(1, 2).contiguous().transpose(1, 2).expand(2, 1, 16, 64)[:, :, ::2], k[:, :, ::2])
    with pytest.raises(ValueError):
        binding.paged_cache(4, 2, 24, 64, device="cpu")
    cache = binding.paged_cache(4, 1, 16, 64, device="cpu")
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.paged_attn(q, cache, table, lens)
    with pytest.raises(ValueError, match="table"):
        binding.paged_attn(q, cache, table[:1], lens)
    with pytest.raises(ValueError, match="table"):
        binding.paged_attn(q, cache, table.long(), lens)
    with pytest.raises(ValueError, match="lens"):
        binding.paged_attn(q, cache, table, lens[:1])
    with pytest.raises(ValueError, match="q must be"):
        binding.paged_attn(q[0], cache, table, lens)
    with pytest.raises(ValueError, match="cu_seqlens"):
        binding.paged_attn_varlen(q[0], cache, table, lens, torch.zeros(3), 1)
    with pytest.raises(ValueError, match="v must"):
        binding.paged_append(cache, table, torch.zeros(2, 1, 1, 64), torch.zeros(2, 2, 1, 64), lens)
    with pytest.raises(ValueError, match="T must"):
        binding.paged_read(cache, table, None, 0)


def test_an_oversized_window_or_sink_stays_out_of_range_or_means_all():
    cache = binding.paged_cache(4, 1, 16, 64, device="cpu")
    full = binding.paged_attn_workspace_bytes(cache, 1, 1, 4, 40)
    assert binding.paged_attn_workspace_bytes(cache, 1, 1, 4, 40, window=1 << 40, n_sink=1 << 40) == full
    for bad in (dict(window=-(1 << 40)), dict(n_sink=-1)):
        with pytest.raises(binding.RingAttnError, match="out of range"):
            binding.paged_attn_workspace_bytes(cache, 1, 1, 4, 40, **bad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_cache_follows_its_memory_and_can_be_copied(dtype):
    """Memory given back and taken again lies elsewhere; copies have their own."""
    cache = binding.paged_cache(4, 2, 16, 64, dtype=dtype, device="cpu")

    def pointers(c):
        return binding._PAGES.unpack(c._c())[:4]

    want = [t.data_ptr() for t in cache] + [0] * (4 - len(cache))
    assert list(pointers(cache)) == want
    cache.v.set_(torch.zeros_like(cache.v))
    assert pointers(cache)[0] == want[0] and pointers(cache)[1] == cache.v.data_ptr() != want[1]
    assert binding._PAGES.unpack(cache._c())[4:] == (4, 2, 16, 64, {torch.bfloat16: 0}.get(dtype, 2))
    other = copy.deepcopy(cache)
    assert type(other) is binding.PagedCache and other.dims == cache.dims and other.dtype == dtype
    assert not set(pointers(other)) & set(pointers(cache)) - {0}
