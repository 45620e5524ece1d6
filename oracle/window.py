"""Attention with a sliding window and a few first tokens that stay visible,
from its definition, float64 NumPy.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Query i sees the keys A(i) = {j <= i : j > i - window or j < n_sink}; the rest
is softmax attention and its chain rule:

    s_ij = scale <q_i, k_j>,  lse_i = log sum_{A(i)} exp(s_ij)
    p_ij = exp(s_ij - lse_i), o_i = sum p_ij v_j
    dv_j = sum_i p_ij do_i,   ds_ij = p_ij (<do_i, v_j> - <do_i, o_i>)
    dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
"""

import numpy as np

from .attention import f64


def allowed(i, j, window, n_sink):
    """Mask [len(i), len(j)] of positions."""
    i, j = np.asarray(i)[:, None], np.asarray(j)[None, :]
    return (j <= i) & ((j > i - window) | (j < n_sink))


def _head(q, k, v, see, scale):
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(axis=1, keepdims=True)
    return e / z, (m + np.log(z))[:, 0]


def window_attention(q, k, v, window, n_sink, scale):
    """q [B,S,H_q,D], k, v [B,S,H_kv,D] -> (out [B,S,H_q,D], lse [B,H_q,S])."""
    q, k, v = f64(q), f64(k), f64(v)
    B, S, H_q, _ = q.shape
    grp = H_q // k.shape[2]
    see = allowed(np.arange(S), np.arange(S), window, n_sink)
    out, lse = np.zeros_like(q), np.zeros((B, H_q, S))
    for b in range(B):
        for h in range(H_q):
            p, lse[b, h] = _head(q[b, :, h], k[b, :, h // grp], v, see, scale)
            out[b, :, h] = p @ v[b, :, h // grp]
    return out, lse


def window_backward(q, k, v, dout, window, n_sink, scale):
    """(dq, dk, dv) of ``window_attention`` for the upstream gradient dout."""
    q, k, v, dout = f64(q), f64(k), f64(v), f64(dout)
    B, S, H_q, _ = q.shape
    grp = H_q // k.shape[2]
    see = allowed(np.arange(S), np.arange(S), window, n_sink)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        for h in range(H_q):
            g = h // grp
            p, _ = _head(q[b, :, h], k[b, :, g], v, see, scale)
            do = dout[b, :, h]
            dv[b, :, g] += p.T @ do
            ds = p * (do @ v[b, :, g].T - (do * (p @ v[b, :, g])).sum(1, keepdims=True))
            dq[b, :, h] = scale * ds @ k[b, :, g]
            dk[b, :, g] += scale * ds.T @ q[b, :, h]
    return dq, dk, dv


def _packed(fn, tensors, cu, *args):
    parts = []
    for a, b in zip(cu[:-1], cu[1:]):
        if b > a:
            parts.append(fn(*[f64(t)[None, a:b] for t in tensors], *args))
    return parts


def window_attention_varlen(q, k, v, cu, window, n_sink, scale):
    """Packed sequences: q [total,H_q,D] -> (out, lse [H_q,total])."""
    parts = _packed(window_attention, (q, k, v), cu, window, n_sink, scale)
    return (np.concatenate([p[0][0] for p in parts]),
            np.concatenate([p[1][0] for p in parts], axis=1))


def window_backward_varlen(q, k, v, dout, cu, window, n_sink, scale):
    parts = _packed(window_backward, (q, k, v, dout), cu, window, n_sink, scale)
    return tuple(np.concatenate([p[i][0] for p in parts]) for i in range(3))
