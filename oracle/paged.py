"""The paged key/value cache from its definition, in NumPy.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Slot j of sequence b is row j % page of page table[b][j // page]; an entry
outside the pool is a page that is not there. In 8 bits a row keeps e4m3 codes
c, 2^e as the byte e + 127, and stands for c 2^e. All float64.
"""

import numpy as np

from .attention import f64


def e4m3_values():
    """The value of each of the 256 codes: sign, 4 bits of exponent (bias 7),
    3 of mantissa; 0x7f and 0xff are NaN, nothing is infinite."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


def quantise(x):
    """(codes uint8 [..., D], bytes uint8 [...]) of rows x [..., D]: the nearest
    code of x / 2^e, of two as near the one with an even mantissa."""
    x = f64(x)
    table = e4m3_values()[:127]                  # 0 up to 448, ascending
    mid = (table[1:] + table[:-1]) / 2
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -117)
    for i, t in np.ndenumerate(top):
        while t / 2.0 ** e[i] > 448.0:
            e[i] += 1
    y = x / 2.0 ** e[..., None].astype(np.float64)
    a = np.where(np.isfinite(y), np.abs(y), 0.0)
    lo = np.searchsorted(mid, a, side="left")    # ties go down here
    tie = np.isin(a, mid)
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8), (e + 127).astype(np.uint8)


def values(codes, byte):
    return e4m3_values()[codes] * 2.0 ** (np.asarray(byte, np.float64) - 127)[..., None]


def there(table, n_pages, page, n):
    """[B, n]: which of the first n slots have a page."""
    table = np.asarray(table)
    at = np.arange(n) // page
    ok = at < table.shape[1]
    ids = table[:, np.minimum(at, table.shape[1] - 1)]
    return ok & (ids >= 0) & (ids < n_pages)


def rows(pool, table, n):
    """The first n slots' rows [B, H_kv, n, ...] of pool [N, H_kv, page, ...];
    those without a page are page 0's."""
    page = pool.shape[2]
    j = np.arange(n)
    ok = there(table, pool.shape[0], page, n)
    ids = np.where(ok, np.asarray(table)[:, np.minimum(j // page, np.shape(table)[1] - 1)], 0)
    return np.moveaxis(pool[ids, :, j % page], 2, 1)


def attention(q, k, v, lens, news, has, window=0, n_sink=0, scale=None):
    """q: one [n_b, H_q, D] a sequence; k, v [B, H_kv, L, D] values; news[b] new
    tokens at the end of lens[b] slots; has [B, L]. Lists of out [n_b, H_q, D],
    lse [H_q, n_b]."""
    outs, lses = [], []
    for b, x in enumerate(q):
        x = f64(x)
        n_b, H_q, D = x.shape
        grp = H_q // k.shape[1]
        s = 1.0 / np.sqrt(D) if scale is None else scale
        out, lse = np.zeros(x.shape), np.full((H_q, n_b), -np.inf)
        for t in range(n_b):
            p = int(lens[b]) - int(news[b]) + t
            j = np.arange(k.shape[2])
            see = (j <= p) & has[b]
            if window > 0:
                see &= (j > p - window) | (j < n_sink)
            see = np.flatnonzero(see)
            if see.size == 0:
                continue
            for h in range(H_q):
                z = s * (k[b, h // grp, see] @ x[t, h])
                m = z.max()
                w = np.exp(z - m)
                lse[h, t] = m + np.log(w.sum())
                out[t, h] = (w / w.sum()) @ v[b, h // grp, see]
        outs.append(out)
        lses.append(lse)
    return outs, lses
