"""Refusals of the 4-bit cache's entry points, before anything reaches a GPU."""

import ctypes

import pytest
import torch

from sequence_exact_attention_gb300 import binding

OK, NULL, SHAPE, HEADDIM, ALIGN, DTYPE, BUFFER, RANGE = 0, 1, 2, 3, 4, 5, 9, 10
A = 0x10000000          # a 16-byte aligned fake address, never dereferenced
vp = ctypes.c_void_p


def addr(i):            # apart by more than any tensor below
    return vp(A + (i << 36))


def append(lib, k=1, v=2, c=(3, 4, 5, 6), start=7, n_new=0, B=2, T=3, H=2, D=64, C=64, dtype=0, off=0):
    return lib.kv4_append(vp(addr(k).value + off) if k else vp(0), addr(v) if v else vp(0),
                          *(addr(x) if x else vp(0) for x in c), addr(start) if start else vp(0),
                          addr(n_new) if n_new else vp(0), B, T, H, D, C, dtype, None, None)


def test_append_refusals(lib):
    assert append(lib, k=0) == NULL and append(lib, v=0) == NULL and append(lib, start=0) == NULL
    assert append(lib, c=(3, 4, 5, 0)) == NULL
    for bad in (dict(B=0), dict(T=0), dict(H=0), dict(C=0), dict(C=24), dict(T=-1)):
        assert append(lib, **bad) == SHAPE, bad
    assert append(lib, D=96) == HEADDIM
    assert append(lib, off=8) == ALIGN
    assert append(lib, dtype=2) == DTYPE
    assert append(lib, B=1 << 16, T=1 << 12, H=8, D=128) == RANGE


def read(lib, k=7, v=8, c=(3, 4, 5, 6), T=3, D=64, C=64, dtype=0):
    return lib.kv4_read(*(addr(x) if x else vp(0) for x in c), None, addr(k) if k else vp(0),
                        addr(v) if v else vp(0), 2, T, 2, D, C, dtype, None, None)


def test_read_refusals(lib):
    assert read(lib, k=0, v=0) == NULL and read(lib, c=(0, 4, 5, 6)) == NULL
    assert read(lib, T=0) == SHAPE and read(lib, C=8) == SHAPE
    assert read(lib, D=32) == HEADDIM and read(lib, dtype=9) == DTYPE


def attn(lib, q=1, c=(3, 4, 5, 6), lens=7, out=8, lse=9, score=0, B=2, S_q=1, H_q=4, H_kv=2, D=64, C=4096,
         max_len=4096, window=0, n_sink=0, dtype=0, ws=10, ws_bytes=1 << 30, off=0):
    p = lambda x: addr(x) if x else vp(0)         # noqa: E731
    return lib.kv4_attn(vp(p(q).value + off) if q else vp(0), *(p(x) for x in c), p(lens), p(out), p(lse), p(score),
                        B, S_q, H_q, H_kv, D, C, max_len, window, n_sink, 0.0, dtype, p(ws), ws_bytes, None, None)


def need(lib, *sizes):
    n = ctypes.c_size_t()
    st = lib.kv4_attn_workspace(*sizes, ctypes.byref(n))
    return st, n.value


def test_attn_refusals(lib):
    for bad in (dict(q=0), dict(lens=0), dict(out=0), dict(c=(3, 0, 5, 6))):
        assert attn(lib, **bad) == NULL, bad
    for bad in (dict(B=0), dict(S_q=0), dict(H_q=3), dict(H_kv=0), dict(C=4090, max_len=100)):
        assert attn(lib, **bad) == SHAPE, bad
    assert attn(lib, D=256) == HEADDIM
    assert attn(lib, dtype=1) == DTYPE                     # bf16 only
    assert attn(lib, off=4) == ALIGN
    for bad in (dict(max_len=0), dict(max_len=4097), dict(window=-1), dict(n_sink=-1),
                dict(B=1 << 15, S_q=1 << 10, H_q=16, H_kv=16, D=128)):
        assert attn(lib, **bad) == RANGE, bad
    st, n = need(lib, 2, 1, 4, 2, 64, 4096, 4096, 0, 0, 0)
    assert st == OK and n > 0
    assert attn(lib, ws_bytes=n - 1) == BUFFER
    assert attn(lib, ws=0) == NULL
    st, m = need(lib, 2, 1, 4, 2, 64, 4096, 4096, 0, 0, 1)
    assert st == OK and m > n                              # scores keep the logits
    assert attn(lib, score=11, ws_bytes=m - 1) == BUFFER


def test_buffers_that_overlap_are_refused(lib):
    for bad in (dict(k=3), dict(v=6), dict(start=4), dict(n_new=5), dict(c=(3, 4, 3, 6))):
        assert append(lib, **bad) == BUFFER, bad
    for bad in (dict(k=3), dict(v=6), dict(k=7, v=7)):
        assert read(lib, **bad) == BUFFER, bad
    for bad in (dict(out=1), dict(out=5), dict(lse=7), dict(score=4), dict(score=8), dict(ws=1), dict(ws=8),
                dict(ws=11, score=11)):
        assert attn(lib, **bad) == BUFFER, bad
    for bad in (dict(dst=(7, 8, 7, 10)), dict(dscore=13), dict(dlens=13)):
        assert evict(lib, **bad) == BUFFER, bad


def test_attn_workspace(lib):
    assert lib.kv4_attn_workspace(2, 1, 4, 2, 64, 4096, 4096, 0, 0, 0, None) == NULL
    assert need(lib, 1, 1, 8, 2, 64, 256, 201, 0, 0, 0) == (OK, 0)       # one chunk, nothing to join
    # a window bounds what is read, and with it the chunks
    wide = need(lib, 1, 1, 8, 2, 128, 1 << 20, 1 << 20, 0, 0, 0)[1]
    assert 0 < need(lib, 1, 1, 8, 2, 128, 1 << 20, 1 << 20, 4096, 4, 0)[1] < wide
    # a window as long as the axis is none
    assert need(lib, 1, 1, 8, 2, 128, 1 << 20, 1 << 20, 1 << 20, 4, 0)[1] == wide
    assert need(lib, 1, 1, 8, 3, 128, 256, 256, 0, 0, 0)[0] == SHAPE
    assert need(lib, 1, 1, 8, 2, 128, 256, 300, 0, 0, 0)[0] == RANGE


def evict(lib, src=(1, 2, 3, 4), score=5, lens=6, dst=(7, 8, 9, 10), dscore=11, dlens=12, kept=13, B=2, H=2, D=64,
          C=4096, C_dst=64, budget=64, sink=4, recent=8):
    p = lambda x: addr(x) if x else vp(0)         # noqa: E731
    return lib.kv4_evict(*(p(x) for x in src), p(score), p(lens), *(p(x) for x in dst), p(dscore), p(dlens), p(kept),
                         B, H, D, C, C_dst, budget, sink, recent, None, None)


def test_evict_refusals(lib):
    for bad in (dict(score=0), dict(lens=0), dict(dlens=0), dict(kept=0), dict(src=(1, 0, 3, 4)),
                dict(dst=(7, 8, 9, 0))):
        assert evict(lib, **bad) == NULL, bad
    for bad in (dict(B=0), dict(H=0), dict(C=100), dict(C_dst=72)):
        assert evict(lib, **bad) == SHAPE, bad
    assert evict(lib, D=80) == HEADDIM
    for bad in (dict(budget=0), dict(budget=65), dict(sink=-1), dict(recent=-1), dict(sink=30, recent=35)):
        assert evict(lib, **bad) == RANGE, bad
    # nothing written may be part of what is read
    for bad in (dict(dst=(1, 8, 9, 10)), dict(dst=(7, 8, 9, 4)), dict(dscore=5), dict(dlens=6), dict(kept=5)):
        assert evict(lib, **bad) == BUFFER, bad


def test_binding_refuses_wrong_tensors():
    f32, i32 = torch.float32, torch.int32
    with pytest.raises(ValueError, match="multiple of 16"):
        binding.kv4_cache(1, 1, 24, 64, "cpu")
    cache = binding.kv4_cache(2, 2, 32, 64, "cpu")
    k = torch.zeros(2, 3, 2, 64)
    lens = torch.zeros(2, dtype=i32)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    cases = [
        (lambda: binding.kv4_append(cache, k, k[:, :2], lens), "v must have shape"),
        (lambda: binding.kv4_append(cache, k[..., :32], k, lens), "k must have shape"),
        (lambda: binding.kv4_append(cache, k, k, lens.long()), "start must be"),
        (lambda: binding.kv4_append(cache, k, k, lens[:1]), "start must have shape"),
        (lambda: binding.kv4_append(cache, k.half(), k.half(), lens), "unsupported dtype"),
        (lambda: binding.KV4Cache(*cache[:3], cache.v_meta.float()), "v_meta must be"),
        (lambda: binding.KV4Cache(cache.k_codes[..., :16], *cache[1:]), "v_codes must have shape"),
        (lambda: binding.KV4Cache(cache.k_codes[0], *cache[1:]), "k_codes must be"),
        (lambda: binding.KV4Cache(cache.k_codes.transpose(0, 1), *cache[1:]), "k_codes must be contiguous"),
        (lambda: binding.kv4_read(cache, lens, 0), "T must be"),
        (lambda: binding.kv4_read(cache, lens, 2, k=torch.zeros(2, 3, 2, 64)), "k must have shape"),
        (lambda: binding.kv4_attn(q[:1], cache, lens), "q must be"),
        (lambda: binding.kv4_attn(q, cache, lens, lse=torch.zeros(2, 1, 4)), "lse must have shape"),
        (lambda: binding.kv4_attn(q, cache, lens, score=torch.zeros(2, 2, 16)), "score must have shape"),
        (lambda: binding.kv4_attn(q, cache, lens, workspace=torch.zeros(4, dtype=f32)), "workspace"),
        (lambda: binding.kv4_evict(cache, torch.zeros(2, 2, 32), lens, 0), "budget"),
        (lambda: binding.kv4_evict(cache, torch.zeros(2, 2, 16), lens, 8), "score must have shape"),
        (lambda: binding.kv4_evict(cache, torch.zeros(2, 2, 32), lens, 8,
                                   dst=binding.kv4_cache(2, 1, 16, 64, "cpu")), "dst must have"),
        # right shapes, but host tensors: no CPU path
        (lambda: binding.kv4_append(cache, k, k, lens), "CUDA tensors"),
        (lambda: binding.kv4_read(cache, lens, 2), "CUDA tensors"),
        (lambda: binding.kv4_attn(q, cache, lens), "CUDA tensors"),
        (lambda: binding.kv4_evict(cache, torch.zeros(2, 2, 32), lens, 8), "CUDA tensors"),
    ]
    for call, text in cases:
        with pytest.raises(ValueError, match=text):
            call()
