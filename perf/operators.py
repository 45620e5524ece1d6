"""What the windowed attention and the 4-bit key/value cache are measured on.

Four passes, each as a user's program makes it:

* ``win_fwd``   attention with a sliding window and a few first tokens that
                stay visible, forward: every query sees itself, the
                ``window - 1`` tokens before it and the first ``sink`` tokens.
* ``win_step``  the same, forward and backward (a training step's share).
* ``kv4_step``  serving: the new tokens' keys and values are appended to a
                cache held in 4 bits, read back (the values the cache now
                holds for them), and the new queries attend to the cache;
                with ``score`` the attention weight that every slot received
                is added to its running sum.
* ``kv4_evict`` the cache is cut down to ``budget`` slots a sequence: the
                first ``sink`` and last ``recent`` slots and, of the others,
                those with the largest accumulated weight.

The 4-bit format: a row of D values (one token, one key/value head) is cut
into groups of 64 along D. A group stores a scale and a zero point in
bfloat16 and 64 codes of 4 bits, dimension 2i in the low and 2i + 1 in the
high half of byte i; a code c stands for scale * (c - 8) + zero.
"""

import math

import torch

own = False

_GROUP = 64
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short prompt of a small head count: launch latency
        {"name": "win_fwd_s256", "op": "win_fwd", "dtype": "bf16", "lengths": "256", "hq": 2, "hkv": 2,
         "d": 64, "window": 64, "sink": 4, "p": 1, "order": "contiguous"},
        # the exact float32 path on an odd length, window and sink count
        {"name": "win_fwd_f32_s777", "op": "win_fwd", "dtype": "f32", "lengths": "777,777", "hq": 4, "hkv": 2,
         "d": 64, "window": 100, "sink": 7, "p": 1, "order": "contiguous"},
        # a long prompt with grouped heads, cut into the halves of 8 ranks
        {"name": "win_fwd_s32k", "op": "win_fwd", "dtype": "bf16", "lengths": "32768", "hq": 32, "hkv": 8,
         "d": 128, "window": 4096, "sink": 4, "p": 8, "order": "zigzag"},
        # an ordinary training step of two sequences
        {"name": "win_step_s4k", "op": "win_step", "dtype": "bf16", "lengths": "4096,4096", "hq": 16, "hkv": 16,
         "d": 128, "window": 1024, "sink": 4, "p": 1, "order": "contiguous"},
        # a packed batch of very different lengths, an empty and a one-token sequence among them
        {"name": "win_step_packed", "op": "win_step", "dtype": "bf16", "lengths": "3000,0,1000,1,777,2222", "hq": 8,
         "hkv": 2, "d": 64, "window": 500, "sink": 16, "p": 1, "order": "contiguous"},
        # a long sequence's training step with grouped heads
        {"name": "win_step_s16k", "op": "win_step", "dtype": "bf16", "lengths": "16384", "hq": 32, "hkv": 8,
         "d": 128, "window": 2048, "sink": 4, "p": 1, "order": "contiguous"},
        # one chat of a few hundred tokens, one new token: latency
        {"name": "kv4_step_b1", "op": "kv4_step", "b": 1, "t": 1, "hq": 8, "hkv": 2, "d": 64, "cap": 256, "ctx": 201,
         "ragged": False, "window": 0, "sink": 0, "score": False},
        # a served batch of different lengths whose slots are scored for eviction
        {"name": "kv4_step_b16_8k", "op": "kv4_step", "b": 16, "t": 1, "hq": 32, "hkv": 8, "d": 128, "cap": 8192,
         "ctx": 8191, "ragged": True, "window": 0, "sink": 0, "score": True},
        # long contexts: the cache is what the step reads
        {"name": "kv4_step_b8_128k", "op": "kv4_step", "b": 8, "t": 1, "hq": 32, "hkv": 8, "d": 128, "cap": 131072,
         "ctx": 131072, "ragged": False, "window": 0, "sink": 0, "score": False},
        # four drafted tokens checked at once over a windowed cache
        {"name": "kv4_verify_window", "op": "kv4_step", "b": 4, "t": 4, "hq": 16, "hkv": 4, "d": 128, "cap": 32768,
         "ctx": 30001, "ragged": True, "window": 4096, "sink": 4, "score": False},
        # a small cache that has just gone over its budget
        {"name": "kv4_evict_b1", "op": "kv4_evict", "b": 1, "hkv": 2, "d": 64, "cap": 512, "ctx": 401, "ragged": False,
         "budget": 256, "sink": 4, "recent": 64},
        # a served batch cut down to an eighth of its long contexts
        {"name": "kv4_evict_b8_32k", "op": "kv4_evict", "b": 8, "hkv": 8, "d": 128, "cap": 32768, "ctx": 32768,
         "ragged": True, "budget": 4096, "sink": 4, "recent": 1024},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["win_fwd", "win_step", "kv4_step", "kv4_evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    grp = rng.choice([1, 2, 4, 8])
    if op in ("win_fwd", "win_step"):
        dtype = "f32" if op == "win_fwd" and rng.random() < 0.25 else "bf16"
        total = _log_uniform(rng, 64, 2048 if dtype == "f32" else 16384)
        n = rng.choice([1, 1, 2, 3, 5])
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lengths = [y - x for x, y in zip([0] + cuts, cuts + [total])]
        if rng.random() < 0.4:                  # a batch of equal lengths
            lengths = [max(1, total // n)] * n
        return {"op": op, "dtype": dtype, "lengths": ",".join(map(str, lengths)), "hq": min(hkv * grp, 32), "hkv": hkv,
                "d": d, "window": _log_uniform(rng, 1, 2048), "sink": rng.choice([0, 1, 4, 5, 64, 200]),
                "p": rng.choice([1, 1, 2, 3, 8]), "order": rng.choice(["contiguous", "zigzag"])}
    cap = 16 * _log_uniform(rng, 4, 4096)
    c = {"op": op, "b": _log_uniform(rng, 1, 12), "hkv": hkv, "d": d, "cap": cap, "ragged": rng.random() < 0.7}
    if op == "kv4_step":
        t = rng.choice([1, 1, 1, 2, 3, 4, 7])
        windowed = rng.random() < 0.4
        return {**c, "t": t, "hq": hkv * grp, "ctx": rng.randint(max(t, cap // 2), cap),
                "window": _log_uniform(rng, 16, 8192) if windowed else 0,
                "sink": rng.choice([0, 4, 33]) if windowed else 0, "score": rng.random() < 0.5}
    budget = 16 * rng.randint(1, cap // 16)
    sink = min(rng.choice([0, 1, 4, 16]), budget)
    return {**c, "ctx": rng.randint(cap // 2, cap), "budget": budget, "sink": sink,
            "recent": rng.randint(0, budget - sink)}


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def _contexts(case):
    """Slots used by each sequence; ragged batches go down to a quarter."""
    least = case.get("t", 1)
    if not case["ragged"]:
        return [case["ctx"]] * case["b"]
    return [max(least, case["ctx"] - (case["ctx"] * 3 * i) // (4 * max(1, case["b"] - 1)))
            for i in range(case["b"])]


def _fixed(case):
    """Sequences of one length come as a batch, others packed."""
    n = _lengths(case)
    return n[0] > 0 and all(x == n[0] for x in n)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] in ("win_fwd", "win_step"):
        n, hq, hkv, d = _lengths(case), case["hq"], case["hkv"], case["d"]
        rows = (len(n), n[0]) if _fixed(case) else (sum(n),)
        dt = _TYPES[case["dtype"]]
        s = {"case": case, "q": normal(*rows, hq, d).to(dt), "k": normal(*rows, hkv, d).to(dt),
             "v": normal(*rows, hkv, d).to(dt)}
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if case["op"] == "win_step":
            s["dout"] = normal(*rows, hq, d).to(dt)
        return s

    b, hkv, d, cap = case["b"], case["hkv"], case["d"], case["cap"]
    lens = torch.tensor(_contexts(case), dtype=torch.int32, device=dev)
    cache = []
    for _ in range(2):          # keys, values: codes of bell-shaped values, scales and zero points around theirs
        shape = (b, hkv, cap, d // 2)
        lo, hi = (normal(*shape).mul_(2.7).add_(8.0).round_().clamp_(0, 15).to(torch.uint8) for _ in range(2))
        scale = (0.3 * (1 + 0.2 * normal(b, hkv, cap, d // _GROUP)).abs_() + 0.02)
        zero = 0.2 * normal(b, hkv, cap, d // _GROUP)
        cache += [lo + hi * 16, torch.stack([scale, zero], -1).to(torch.bfloat16)]
    s = {"case": case, "cache": cache, "lens": lens}
    if case["op"] == "kv4_step":
        t = case["t"]
        s["q"] = normal(b, t, case["hq"], d).to(torch.bfloat16)
        s["k"] = normal(b, t, hkv, d).to(torch.bfloat16)
        s["v"] = normal(b, t, hkv, d).to(torch.bfloat16)
        s["start"] = lens - t
        if case["score"]:
            s["score"] = normal(b, hkv, cap).exp_()
    else:
        # a few sums tie, as sums of many near-zero weights do
        s["score"] = normal(b, hkv, cap).mul_(2.0).exp_().to(torch.bfloat16).float()
        n = case["budget"]
        s["dst"] = [torch.zeros(b, hkv, n, *x.shape[3:], dtype=x.dtype, device=dev) for x in cache]
        s["dst_score"] = torch.zeros(b, hkv, n, device=dev)
        s["zero"] = torch.zeros(b, dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "win_fwd":
        return _window_plain(state, case, None)
    if case["op"] == "win_step":
        return _window_plain(state, case, state["dout"])
    if case["op"] == "kv4_step":
        return _step_plain(state, case)
    return _evict_plain(state, case)


def _own(s, case):
    from sequence_exact_attention_gb300 import binding as ra

    if case["op"] in ("win_fwd", "win_step"):
        q, k, v = s["q"], s["k"], s["v"]
        window, sink, p, order = case["window"], case["sink"], case["p"], case["order"]
        if _fixed(case):
            out, lse = ra.ring_attn_fwd_window(q, k, v, p, window, sink, order=order)
            if case["op"] == "win_fwd":
                return out, lse
            return (out, lse, *ra.ring_attn_bwd_window(q, k, v, out, lse, s["dout"], p, window, sink, order=order))
        longest = max(_lengths(case))
        out, lse = ra.ring_attn_fwd_window_varlen(q, k, v, s["cu"], longest, p, window, sink, order=order)
        if case["op"] == "win_fwd":
            return out, lse
        return (out, lse, *ra.ring_attn_bwd_window_varlen(q, k, v, out, lse, s["dout"], s["cu"], longest, p, window,
                                                          sink, order=order))
    cache = ra.KV4Cache(*s["cache"])
    if case["op"] == "kv4_step":
        ra.kv4_append(cache, s["k"], s["v"], s["start"])
        k, v = ra.kv4_read(cache, s["start"], case["t"])
        out, lse = ra.kv4_attn(s["q"], cache, s["lens"], window=case["window"], n_sink=case["sink"],
                               score=s.get("score"))
        return (out, lse, k, v) + ((s["score"],) if case["score"] else ())
    dst = ra.KV4Cache(*s["dst"])
    dst, score, lens, kept = ra.kv4_evict(cache, s["score"], s["lens"], case["budget"], case["sink"], case["recent"],
                                          dst=dst, dst_score=s["dst_score"])
    return (*ra.kv4_read(dst, s["zero"], case["budget"]), score, lens, kept)


# ---- plain forms

def _window_plain(s, case, dout):
    """Queries in blocks against the strip of keys their windows span, and
    against every sequence's first tokens, each row masked to its own."""
    dt, d, hkv = _TYPES[case["dtype"]], case["d"], case["hkv"]
    grp = case["hq"] // hkv
    cu = s["cu"].long()
    q, k, v = (s[x].reshape(-1, s[x].shape[-2], d).float() for x in "qkv")
    n, dev = q.shape[0], q.device
    window, sink = min(case["window"], n), case["sink"]
    scale = 1.0 / math.sqrt(d)
    bs = min(512, n)
    nb, strip = -(-n // bs), window - 1 + bs
    pad = nb * bs - n

    def blocks(x):              # [n, hq, d] -> [nb, hkv, grp * bs, d]
        x = torch.cat([x, x.new_zeros(pad, *x.shape[1:])]).view(nb, bs, hkv, grp, d)
        return x.permute(0, 2, 3, 1, 4).reshape(nb, hkv, grp * bs, d)

    def rows(x):                # and back
        return x.view(nb, hkv, grp, bs, d).permute(0, 3, 1, 2, 4).reshape(nb * bs, hkv * grp, d)[:n]

    at = torch.arange(nb, device=dev)[:, None] * bs
    i = at + torch.arange(bs, device=dev)                          # [nb, bs]
    j = at - (window - 1) + torch.arange(strip, device=dev)        # [nb, strip]
    seq = torch.bucketize(torch.arange(n, device=dev), cu[1:], right=True)
    iv, jv = i.clamp(max=n - 1), j.clamp(0, n - 1)
    ii, jj = i[:, :, None], j[:, None, :]
    see = (jj <= ii) & (jj > ii - window) & (jj >= 0) & (jj < n) & (seq[iv][:, :, None] == seq[jv][:, None, :])
    kb, vb = (x[jv].permute(0, 2, 1, 3) for x in (k, v))           # [nb, hkv, strip, d]
    qb = blocks(q)
    # columns for every sequence's first tokens, for rows whose window has left them behind
    first = (cu[:-1, None] + torch.arange(sink, device=dev)).reshape(-1)
    owner = torch.arange(cu.numel() - 1, device=dev).repeat_interleave(sink)
    real = (first < cu[1:][owner]) & (first < n)
    fv = first.clamp(max=n - 1)
    far = (seq[iv][:, :, None] == owner) & (first <= ii - window) & real
    ks, vs = (x[fv].permute(1, 0, 2) for x in (k, v))              # [hkv, columns, d]

    see = torch.cat([see, far], -1)[:, None, None].expand(nb, hkv, grp, bs, -1).reshape(nb, hkv, grp * bs, -1)
    z = torch.cat([qb @ kb.transpose(-1, -2), qb @ ks.transpose(-1, -2)], -1)
    z.mul_(scale).masked_fill_(~see, -math.inf)
    top = z.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total.clamp(min=1.0))      # a row that sees a key sums to 1 or more; rows past the last to 0
    o = p[..., :strip] @ vb + p[..., strip:] @ vs
    out = rows(o).to(dt).view_as(s["q"])
    lse = (top + total.log()).view(nb, hkv, grp, bs).permute(1, 2, 0, 3).reshape(case["hq"], nb * bs)[:, :n]
    if _fixed(case):
        lse = lse.view(case["hq"], len(_lengths(case)), -1).transpose(0, 1)
    lse = lse.contiguous()
    if dout is None:
        return out, lse

    do = blocks(dout.reshape(n, case["hq"], d).float())

    def spread(x_strip, x_first):
        r = torch.zeros(n, hkv, d, device=dev)
        r.index_add_(0, jv.reshape(-1), x_strip.permute(0, 2, 1, 3).reshape(-1, hkv, d))
        return r.index_add_(0, fv, x_first.permute(1, 0, 2))

    dv = spread(p[..., :strip].transpose(-1, -2) @ do, (p[..., strip:].transpose(-1, -2) @ do).sum(0))
    dp = torch.cat([do @ vb.transpose(-1, -2), do @ vs.transpose(-1, -2)], -1)
    ds = dp.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dk = spread(ds[..., :strip].transpose(-1, -2) @ qb, (ds[..., strip:].transpose(-1, -2) @ qb).sum(0))
    dq = rows(ds[..., :strip] @ kb + ds[..., strip:] @ ks)
    return (out, lse, (dq * scale).to(dt).view_as(s["q"]), (dk * scale).to(dt).view_as(s["k"]),
            dv.to(dt).view_as(s["v"]))


def _values(codes, meta, dtype=torch.float32):
    """What codes [..., d/2] with (scale, zero) [..., d/64, 2] stand for."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(dtype) - 8
    m = meta.to(dtype).repeat_interleave(_GROUP, -2)
    return c * m[..., 0] + m[..., 1]


def _quantise(x):
    """Codes and (scale, zero) of rows [..., d]: steps of a fifteenth of the
    group's range, rounded to bfloat16, around the ninth of sixteen levels."""
    x = x.float().unflatten(-1, (-1, _GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    scale = (hi / 15 - lo / 15).to(torch.bfloat16)
    zero = (lo + 8 * scale.float()).to(torch.bfloat16)
    step = scale.float()[..., None]
    c = torch.where(step > 0, (x - zero.float()[..., None]) / step, torch.zeros_like(x)).round_().clamp_(-8, 7).add_(8)
    c = c.to(torch.uint8).flatten(-2)
    return c[..., 0::2] + c[..., 1::2] * 16, torch.stack([scale, zero], -1)


def _step_plain(s, case):
    b, t, hq, hkv, d, cap = (case[x] for x in ("b", "t", "hq", "hkv", "d", "cap"))
    grp = hq // hkv
    kc, km, vc, vm = s["cache"]
    dev = kc.device
    slot = (s["start"].long()[:, None] + torch.arange(t, device=dev))                # [b, t]
    bi = torch.arange(b, device=dev)[:, None]
    fresh = []
    for codes, meta, x in ((kc, km, s["k"]), (vc, vm, s["v"])):
        c, m = _quantise(x)                                                          # [b, t, hkv, ...]
        codes[bi, :, slot] = c
        meta[bi, :, slot] = m
        fresh.append(_values(c, m).to(torch.bfloat16))
    k, v = _values(kc, km), _values(vc, vm)                                          # [b, hkv, cap, d]
    q = s["q"].float().view(b, t, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * grp, d)
    z = (q @ k.transpose(-1, -2)).view(b, hkv, t, grp, cap).mul_(1.0 / math.sqrt(d))
    j = torch.arange(cap, device=dev)
    at = slot[:, :, None]                                                            # [b, t, 1]
    see = j <= at
    if case["window"]:
        see = see & ((j > at - case["window"]) | (j < case["sink"]))
    z.masked_fill_(~see[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total)
    o = (p.view(b, hkv, t * grp, cap) @ v).view(b, hkv, t, grp, d)
    out = o.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(torch.bfloat16)
    lse = (top + total.log())[..., 0].permute(0, 1, 3, 2).reshape(b, hq, t)
    if not case["score"]:
        return out, lse, *fresh
    s["score"].add_(p.sum((2, 3)))
    return out, lse, *fresh, s["score"]


def _evict_plain(s, case):
    b, hkv, cap, n = case["b"], case["hkv"], case["cap"], case["budget"]
    dev = s["score"].device
    lens = s["lens"].long()[:, None, None]
    j = torch.arange(cap, device=dev)
    rank = torch.where(j < case["sink"], math.inf, s["score"])
    rank = torch.where(j >= lens - case["recent"], math.inf, rank)
    rank = torch.where(j < lens, rank, -math.inf)
    by = rank.sort(dim=-1, descending=True, stable=True).indices[..., :n]                 # the lowest slot first among equals
    left = lens.clamp(max=n)
    kept = torch.where(torch.arange(n, device=dev) < left, by, cap).sort(-1).values   # back in slot order
    gone = kept >= cap
    at = kept.clamp(max=cap - 1)
    for x, y in zip([*s["cache"], s["score"]], [*s["dst"], s["dst_score"]]):
        flat = x.reshape(b, hkv, cap, -1)
        got = flat.gather(2, at[..., None].expand(-1, -1, -1, flat.shape[-1])).view_as(y)
        y.copy_(torch.where(gone.view(b, hkv, n, *[1] * (y.dim() - 3)), y, got))
    k, v = (_values(c, m).to(torch.bfloat16).transpose(1, 2).contiguous() for c, m in (s["dst"][:2], s["dst"][2:]))
    return k, v, s["dst_score"], left.view(b).int(), torch.where(gone, -1, kept).int()


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("win_fwd", "win_step"):
        return _window_exact(s, case)
    if case["op"] == "kv4_step":
        return _step_exact(s, case)
    return _evict_exact(s, case)


def _window_exact(s, case):
    """Sequence by sequence, some rows at a time, every mask from positions."""
    n, hq, hkv, d, w, sink = _lengths(case), case["hq"], case["hkv"], case["d"], case["window"], case["sink"]
    grp, scale, back = hq // hkv, d ** -0.5, case["op"] == "win_step"
    q, k, v = (s[x].reshape(-1, s[x].shape[-2], d).double() for x in "qkv")
    do = s["dout"].reshape(-1, hq, d).double() if back else None
    out, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.zeros(hq, q.shape[0], dtype=torch.float64, device=q.device)
    base = 0
    for length in n:
        for r0 in range(0, length, 256):
            r1 = min(length, r0 + 256)
            lo = max(0, r0 - w + 1)
            pos = torch.tensor(sorted(set(range(min(sink, length, r1))) | set(range(lo, r1))), device=q.device)
            i = torch.arange(r0, r1, device=q.device)[:, None]
            see = (pos <= i) & ((i - pos < w) | (pos < sink))
            for h in range(hkv):
                heads = slice(h * grp, (h + 1) * grp)
                x = q[base + r0:base + r1, heads].transpose(0, 1)                    # [grp, rows, d]
                kk, vv = k[base + pos, h], v[base + pos, h]
                z = torch.where(see, scale * (x @ kk.T), -math.inf)
                norm = torch.logsumexp(z, -1)
                p = torch.exp(z - norm[..., None])
                o = p @ vv
                out[base + r0:base + r1, heads] = o.transpose(0, 1)
                lse[heads, base + r0:base + r1] = norm
                if back:
                    g = do[base + r0:base + r1, heads].transpose(0, 1)
                    ds = p * (g @ vv.T - (g * o).sum(-1, keepdim=True)) * scale
                    dq[base + r0:base + r1, heads] = (ds @ kk).transpose(0, 1)
                    dk[base + pos, h] += torch.einsum("gij,gid->jd", ds, x)
                    dv[base + pos, h] += torch.einsum("gij,gid->jd", p, g)
        base += length
    if _fixed(case):
        lse = lse.view(hq, len(n), -1).transpose(0, 1).contiguous()
    res = (out.view_as(s["q"]), lse)
    return res + ((dq.view_as(s["q"]), dk.view_as(s["k"]), dv.view_as(s["v"])) if back else ())


def _decoded(codes, meta):
    """Value by value: nibble i % 2 of byte i // 2, group i // 64."""
    d = 2 * codes.shape[-1]
    i = torch.arange(d, device=codes.device)
    c = (codes[..., i // 2].to(torch.int16) >> (4 * (i % 2))) & 15
    return meta[..., i // _GROUP, 0].double() * (c.double() - 8) + meta[..., i // _GROUP, 1].double()


def _encoded(x):
    """The value each element of x is held as, in 64 bits; the scale and the
    zero point are rounded to bfloat16 once, from 64 bits."""
    y = x.double().unflatten(-1, (-1, _GROUP))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15).to(torch.bfloat16).double()
    zero = (lo + 8 * scale).to(torch.bfloat16).double()
    c = torch.round((y - zero) / scale.clamp(min=1e-300)).clamp(-8, 7)
    return (c * scale + zero).flatten(-2)


def _step_exact(s, case):
    b, t, hq, hkv, d = (case[x] for x in ("b", "t", "hq", "hkv", "d"))
    grp = hq // hkv
    fresh = [_encoded(s[x]) for x in "kv"]
    out = torch.zeros(b, t, hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(b, hq, t, dtype=torch.float64, device=s["q"].device)
    score = s["score"].double() if case["score"] else None
    for i, n in enumerate(_contexts(case)):
        for h in range(hkv):
            k, v = (_decoded(c[i, h, :n], m[i, h, :n]) for c, m in (s["cache"][:2], s["cache"][2:]))
            k[n - t:], v[n - t:] = fresh[0][i, :, h], fresh[1][i, :, h]
            for r in range(t):
                heads, at = slice(h * grp, (h + 1) * grp), n - t + r
                pos = torch.arange(at + 1, device=k.device)
                if case["window"]:
                    pos = pos[(pos < case["sink"]) | (at - pos < case["window"])]
                z = s["q"][i, r, heads].double() @ k[pos].T * d ** -0.5
                norm = torch.logsumexp(z, -1)
                p = torch.exp(z - norm[:, None])
                out[i, r, heads], lse[i, heads, r] = p @ v[pos], norm
                if score is not None:
                    score[i, h, pos] += p.sum(0)
    return (out, lse, *fresh) + ((score,) if case["score"] else ())


def _evict_exact(s, case):
    b, hkv, d, n = case["b"], case["hkv"], case["d"], case["budget"]
    k, v = (torch.zeros(b, n, hkv, d, dtype=torch.float64, device=s["score"].device) for _ in range(2))
    score = torch.zeros(b, hkv, n, dtype=torch.float64, device=s["score"].device)
    for i, length in enumerate(_contexts(case)):
        for h in range(hkv):
            slots = torch.arange(length, device=score.device)
            if length > n:
                a, z = case["sink"], length - case["recent"]
                a = min(a, z)
                w = s["score"][i, h, a:z].double()
                order = torch.argsort(-w, stable=True)[:n - a - (length - z)]
                slots = torch.cat([slots[:a], a + order.sort().values, slots[z:]])
            m = slots.numel()
            for x, (c, q) in zip((k, v), (s["cache"][:2], s["cache"][2:])):
                x[i, :m, h] = _decoded(c[i, h, slots], q[i, h, slots])
            score[i, h, :m] = s["score"][i, h, slots].double()
    return k, v, score, None, None


# ------------------------------------------------------------------ work

def _pairs(length, window, sink):
    """(query, key) pairs: each query sees min(i + 1, window) tokens up to
    itself and the first tokens that its window has left behind."""
    w = min(window, length)
    band = w * (w + 1) // 2 + (length - w) * w
    f = min(sink, max(0, length - w))
    return band + f * (length - w) - f * (f - 1) // 2


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] in ("win_fwd", "win_step"):
        n, hq = _lengths(case), case["hq"]
        size = 4 if case["dtype"] == "f32" else 2
        total, pairs = sum(n), sum(_pairs(x, case["window"], case["sink"]) for x in n)
        q, kv, lse = total * hq * d * size, total * hkv * d * size, total * hq * 4
        if case["op"] == "win_fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * hq * d * pairs}
        # forward, and backward with its five products
        return {"bytes": 2 * q + 2 * kv + lse + 4 * q + 4 * kv + lse, "flops": 14 * hq * d * pairs}
    row = d // 2 + 4 * (d // _GROUP)                 # bytes of one key or value row
    if case["op"] == "kv4_step":
        t, hq, slots, pairs = case["t"], case["hq"], 0, 0
        for n in _contexts(case):
            seen = [min(n - t + r + 1, case["window"] + case["sink"]) if case["window"] else n - t + r + 1
                    for r in range(t)]
            slots += min(n, seen[-1] + t - 1)
            pairs += sum(seen)
        fresh = case["b"] * t * hkv
        io = case["b"] * t * hq * (4 * d + 4)
        moved = 2 * slots * hkv * row + 2 * fresh * (2 * d + row + 2 * d) + io
        return {"bytes": moved + (8 * slots * hkv if case["score"] else 0), "flops": 4 * hq * d * pairs}
    used = _contexts(case)
    left = sum(min(x, case["budget"]) for x in used)
    out = case["b"] * case["budget"] * 4 * d + left * 2 * row                      # the values read back
    return {"bytes": hkv * (4 * sum(used) + left * (4 * row + 8) + out), "flops": hkv * 4 * d * left}
