"""Refusals of the windowed entry points, before anything reaches a GPU."""

import ctypes

import pytest
import torch

from sequence_exact_attention_gb300 import binding

OK, NULL, SHAPE, HEADDIM, ALIGN, DTYPE, BUFFER, RANGE = 0, 1, 2, 3, 4, 5, 9, 10
A = 0x10000          # a 16-byte aligned fake address, never dereferenced
vp = ctypes.c_void_p


def fwd(lib, q=A, out=A, B=1, H_q=4, H_kv=2, S=1000, D=128, P=2, window=100, n_sink=4, dtype=0, order=0):
    return lib.ring_attn_fwd_window(vp(q), vp(A), vp(A), vp(out), vp(A), B, H_q, H_kv, S, D, P, window, n_sink, 0.0,
                                    dtype, order, None, None)


def fwd_varlen(lib, cu=A, n=3, total=600, mx=300, window=100, n_sink=4, D=128, dtype=0):
    return lib.ring_attn_fwd_window_varlen(*[vp(A)] * 5, vp(cu), n, total, mx, 4, 2, D, 1, window, n_sink, 0.0, dtype,
                                           0, None, None)


def need(lib, B=1, H_q=4, H_kv=2, S=1000, D=128, P=2, window=100, n_sink=4, order=0, varlen=0):
    n = ctypes.c_size_t()
    st = lib.ring_attn_bwd_window_workspace(B, H_q, H_kv, S, D, P, window, n_sink, order, varlen, ctypes.byref(n))
    return st, n.value


def bwd(lib, dout=A, ws=A, ws_bytes=1 << 30, H_q=4, window=100, n_sink=4, dtype=0, D=128):
    return lib.ring_attn_bwd_window(*[vp(A)] * 5, vp(dout), *[vp(A)] * 3, 1, H_q, 2, 1000, D, 2, window, n_sink, 0.0,
                                    dtype, 0, vp(ws), ws_bytes, None, None)


def bwd_varlen(lib, cu=A, n=3, mx=300, window=100, n_sink=4, dtype=0, ws_bytes=1 << 30):
    return lib.ring_attn_bwd_window_varlen(*[vp(A)] * 9, vp(cu), n, 600, mx, 4, 2, 128, 1, window, n_sink, 0.0, dtype,
                                           0, vp(A), ws_bytes, None, None)


def test_forward_refusals(lib):
    assert fwd(lib, q=0) == NULL and fwd(lib, out=0) == NULL
    for bad in (dict(B=0), dict(S=0), dict(H_q=3), dict(P=0)):
        assert fwd(lib, **bad) == SHAPE, bad
    assert fwd(lib, D=96) == HEADDIM and fwd(lib, q=A + 8) == ALIGN
    assert fwd(lib, dtype=2) == DTYPE and fwd(lib, order=2) == DTYPE
    for bad in (dict(window=0), dict(window=-1), dict(n_sink=-1), dict(S=1 << 22, H_q=64, H_kv=64)):
        assert fwd(lib, **bad) == RANGE, bad


def test_packed_forward_refusals(lib):
    assert fwd_varlen(lib, cu=0) == NULL
    assert fwd_varlen(lib, n=0) == SHAPE and fwd_varlen(lib, mx=0) == SHAPE
    assert fwd_varlen(lib, cu=A + 2) == ALIGN and fwd_varlen(lib, D=32) == HEADDIM
    assert fwd_varlen(lib, dtype=3) == DTYPE
    assert fwd_varlen(lib, window=0) == RANGE and fwd_varlen(lib, n_sink=-3) == RANGE


def test_backward_refusals(lib):
    assert bwd(lib, dout=0) == NULL and bwd(lib, ws=0) == NULL
    assert bwd(lib, H_q=3) == SHAPE and bwd(lib, D=80) == HEADDIM
    assert bwd(lib, dtype=1) == DTYPE                       # bf16 only
    assert bwd(lib, dout=A + 8) == ALIGN and bwd(lib, ws=A + 4) == ALIGN
    assert bwd(lib, window=0) == RANGE and bwd(lib, n_sink=-1) == RANGE
    st, n = need(lib)
    assert st == OK and bwd(lib, ws_bytes=n - 1) == BUFFER
    assert bwd_varlen(lib, cu=0) == NULL and bwd_varlen(lib, n=0) == SHAPE
    assert bwd_varlen(lib, dtype=1) == DTYPE and bwd_varlen(lib, window=-2) == RANGE
    st, n = need(lib, B=3, S=300, P=1, varlen=1)
    assert st == OK and bwd_varlen(lib, ws_bytes=n - 1) == BUFFER


def test_workspace(lib):
    assert lib.ring_attn_bwd_window_workspace(1, 4, 2, 1000, 128, 2, 100, 4, 0, 0, None) == NULL
    one = dict(H_q=2, H_kv=2)                              # a query head a key/value head: no heads to share out
    st, rows = need(lib, n_sink=0, **one)
    assert st == OK and rows == binding.bwd_workspace_bytes(1, 2, 1000, 128, 2)     # no parts without first tokens
    # a window that sees everything needs no shares
    assert need(lib, window=1000, **one) == (OK, rows)
    # few key tiles with eight heads each: a part for every head of the 2 x 8 tiles
    st, n = need(lib, H_q=16, n_sink=0)
    assert st == OK and n - binding.bwd_workspace_bytes(1, 16, 1000, 128, 2) == 16 * 8 * (2 * 128 * 128 * 4)
    # ... but not where the key tiles fill the card
    assert need(lib, H_q=16, B=8, S=8000, n_sink=0) == (OK, binding.bwd_workspace_bytes(8, 16, 8000, 128, 1))
    # long sequences: shares of 2 x 128 x D floats for the one tile of every key/value head
    st, n = need(lib, S=100000, P=1)
    base = binding.bwd_workspace_bytes(1, 4, 100000, 128, 1)
    part = 2 * 128 * 128 * 4
    assert n > base and (n - base) % (2 * part) == 0
    assert (n - base) // (2 * part) <= 4 * 152
    for bad in (dict(window=0), dict(n_sink=-1)):
        assert need(lib, **bad)[0] == RANGE
    assert need(lib, S=0)[0] == SHAPE and need(lib, D=48)[0] == HEADDIM


def test_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    q, k = torch.zeros(1, 256, 4, 64, dtype=bf), torch.zeros(1, 256, 2, 64, dtype=bf)
    lse = torch.zeros(1, 4, 256)
    cu = torch.tensor([0, 100, 256], dtype=torch.int32)
    cases = [
        (lambda: binding.ring_attn_fwd_window(q, k[:, :9], k, 1, 64), "k must have shape"),
        (lambda: binding.ring_attn_fwd_window(q, k, k.float(), 1, 64), "v must be"),
        (lambda: binding.ring_attn_fwd_window(q, k, k, 1, 64, out=q.float()), "out must be"),
        (lambda: binding.ring_attn_fwd_window(q, k, k, 1, 64, lse=lse[:, :2]), "lse must have shape"),
        (lambda: binding.ring_attn_fwd_window(q.half(), k.half(), k.half(), 1, 64), "unsupported dtype"),
        (lambda: binding.ring_attn_bwd_window(q, k, k, q, lse, q, 1, 64, dk=q), "dk must have shape"),
        (lambda: binding.ring_attn_bwd_window(q, k, k, q, lse, q, 1, 64, workspace=lse), "workspace"),
        (lambda: binding.ring_attn_fwd_window_varlen(q[0], k[0], k[0], cu.long(), 156, 1, 64), "cu_seqlens"),
        (lambda: binding.ring_attn_bwd_window_varlen(q[0], k[0], k[0], q[0], lse[0], q[0, :9], cu, 156, 1, 64),
         "dout must have shape"),
        # right shapes, but host tensors: no CPU path
        (lambda: binding.ring_attn_fwd_window(q, k, k, 1, 64), "CUDA tensor"),
        (lambda: binding.ring_attn_bwd_window(q, k, k, q, lse, q, 1, 64), "CUDA tensor"),
        (lambda: binding.ring_attn_fwd_window_varlen(q[0], k[0], k[0], cu, 156, 1, 64), "CUDA tensor"),
        (lambda: binding.ring_attn_bwd_window_varlen(q[0], k[0], k[0], q[0], lse[0], q[0], cu, 156, 1, 64),
         "CUDA tensor"),
    ]
    for call, text in cases:
        with pytest.raises(ValueError, match=text):
            call()
