"""The 4-bit key/value cache from its definition, in NumPy.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

A row of D values is cut into groups of 64. A group keeps a scale and a zero
point, both bfloat16, and 64 codes c in 0..15 that stand for
scale * (c - 8) + zero. ``quantise`` follows the rule step by step in float32
(every step is one IEEE operation, so its codes can be asked for exactly);
everything else is float64.
"""

import numpy as np

from .attention import f64

GROUP = 64


def bf16(x):
    """float32 values rounded to bfloat16 (to nearest, half to even)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    odd = (u >> 16) & 1
    r = ((u + 0x7FFF + odd) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def quantise(x):
    """codes [..., D] (0..15), scale and zero [..., D/64] of rows x [..., D]."""
    x = np.asarray(x, dtype=np.float32)
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = y.min(-1), y.max(-1)
    f = np.float32
    with np.errstate(invalid="ignore", divide="ignore"):
        scale = bf16(hi / f(15) - lo / f(15))
        zero = bf16(lo + f(8) * scale)
        bad = ~np.isfinite(y).all(-1)
        scale, zero = np.where(bad, f(np.nan), scale), np.where(bad, f(np.nan), zero)
        n = np.rint((y - zero[..., None]) / scale[..., None])
    n = np.where(scale[..., None] > 0, n, f(0))
    codes = (np.clip(n, -8, 7) + 8).astype(np.uint8)
    return codes.reshape(x.shape), scale, zero


def pack(codes):
    """Two codes a byte: dimension 2i in the low half of byte i."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), dtype=np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def values(codes, scale, zero):
    """What codes [..., D] stand for, float64."""
    s, z = (np.repeat(f64(m), GROUP, axis=-1) for m in (scale, zero))
    return s * (codes.astype(np.float64) - 8.0) + z


def visible(p, n, window, n_sink):
    """Mask over n slots for a query at slot p."""
    j = np.arange(n)
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < n_sink)
    return see


def cache_attention(q, k, v, lens, window=0, n_sink=0, scale=None):
    """Attention of q [B, S_q, H_q, D] over the cache values k, v
    [B, H_kv, C, D]; returns (out, lse [B, H_q, S_q], weight [B, H_kv, C],
    the weights summed over queries and the heads of a group)."""
    q = f64(q)
    B, S_q, H_q, D = q.shape
    H_kv, C = k.shape[1], k.shape[2]
    grp = H_q // H_kv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out = np.zeros((B, S_q, H_q, D))
    lse = np.full((B, H_q, S_q), -np.inf)
    weight = np.zeros((B, H_kv, C))
    for b in range(B):
        n = int(lens[b])
        for t in range(S_q):
            see = np.flatnonzero(visible(n - S_q + t, C, window, n_sink)[:max(n, 0)])
            if see.size == 0:
                continue
            for h in range(H_q):
                s = scale * (k[b, h // grp, see] @ q[b, t, h])
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                lse[b, h, t] = m + np.log(z)
                out[b, t, h] = (e / z) @ v[b, h // grp, see]
                weight[b, h // grp, see] += e / z
    return out, lse, weight


def evict(score, n, budget, n_sink, n_recent):
    """The slots one head keeps of its first n, ascending."""
    if n <= budget:
        return list(range(n))
    middle = range(n_sink, n - n_recent)
    rank = [(-np.inf if np.isnan(score[j]) else float(score[j])) for j in range(n)]
    # NaN below every number, -inf among them
    order = sorted(middle, key=lambda j: (bool(np.isnan(score[j])), -rank[j], j))
    chosen = order[:budget - n_sink - n_recent]
    return sorted(list(range(n_sink)) + chosen + list(range(n - n_recent, n)))
