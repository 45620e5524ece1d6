"""What the paged key/value cache and the attention over it are measured on.

Three passes, each as a serving program makes it:

* ``write``   new tokens' keys and values are written to the pages (rounded to
              bfloat16 or quantised to 8 bits) and the slots that they went to
              are read back.
* ``decode``  one or a few new tokens a sequence: their keys and values are
              appended and read back (the values the pages now hold for them),
              and their queries attend to the pages.
* ``prompt``  the same of a packed batch of pieces of prompts, each behind what
              its sequence's pages already hold.

Pages: ``[N, H_kv, page, D]``; slot j of sequence b is row ``j % page`` of page
``table[b, j // page]``; a table entry below 0 is a page that is not there. In
8 bits a row of D values (one token, one head) is 8-bit floating-point codes
(e4m3) and one power of two 2^e, held as the byte e + 127: the least e from
-117 on with ``max |x| / 2^e <= 448``.

A query at slot p sees the slots j <= p; with a window only those with
j > p - window or j < sink. A window of 0 is none.
"""

import math

import torch

own = False

_CODE = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of a small model: launch latency
        {"name": "write_b1", "op": "write", "pool": "e4m3", "src": "bf16", "new": "1", "ctx": "37", "hkv": 2, "d": 64,
         "page": 16},
        # a batch's ragged prompts in float32 written as bfloat16, one of them empty
        {"name": "write_f32_ragged", "op": "write", "pool": "bf16", "src": "f32", "new": "777,0,1500,33,2001",
         "ctx": "0,5,64,1000,31", "hkv": 4, "d": 64, "page": 32},
        # prompts of a served batch, quantised as they are written
        {"name": "write_8x8k", "op": "write", "pool": "e4m3", "src": "bf16", "new": ",".join(["8192"] * 8),
         "ctx": ",".join(["0"] * 8), "hkv": 8, "d": 128, "page": 64},
        # one chat of a few hundred tokens, one new token: latency
        {"name": "decode_b1", "op": "decode", "pool": "bf16", "b": 1, "t": 1, "hq": 8, "hkv": 2, "d": 64, "page": 16,
         "cap": 256, "ctx": 201, "ragged": False, "window": 0, "sink": 0},
        # a served batch of different lengths
        {"name": "decode_b32_8k", "op": "decode", "pool": "bf16", "b": 32, "t": 1, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "cap": 8192, "ctx": 8191, "ragged": True, "window": 0, "sink": 0},
        # long contexts in 8 bits: the pages are what the step reads
        {"name": "decode_b8_128k", "op": "decode", "pool": "e4m3", "b": 8, "t": 1, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "cap": 131072, "ctx": 131072, "ragged": False, "window": 0, "sink": 0},
        # four drafted tokens checked at once under a window
        {"name": "decode_verify", "op": "decode", "pool": "e4m3", "b": 4, "t": 4, "hq": 16, "hkv": 4, "d": 128,
         "page": 32, "cap": 32768, "ctx": 30001, "ragged": True, "window": 4096, "sink": 4},
        # a short prompt of a small model, nothing cached
        {"name": "prompt_s200", "op": "prompt", "pool": "bf16", "new": "200", "ctx": "0", "hq": 4, "hkv": 2, "d": 64,
         "page": 16, "window": 0, "sink": 0},
        # a packed batch: whole prompts, pieces behind a prefix, a decoding token, an empty place
        {"name": "prompt_packed", "op": "prompt", "pool": "e4m3", "new": "3000,0,1000,1,777,222",
         "ctx": "0,100,2000,4095,513,3001", "hq": 8, "hkv": 2, "d": 64, "page": 64, "window": 0, "sink": 0},
        # a piece of a long prompt
        {"name": "prompt_4k_of_16k", "op": "prompt", "pool": "bf16", "new": "4096", "ctx": "12288", "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "window": 0, "sink": 0},
        # the same of an 8-bit cache under a window, two sequences
        {"name": "prompt_window_8bit", "op": "prompt", "pool": "e4m3", "new": "2048,1500", "ctx": "9000,6001", "hq": 16,
         "hkv": 4, "d": 128, "page": 32, "window": 2048, "sink": 4},
        # a short question behind a long document
        {"name": "prompt_64_of_100k", "op": "prompt", "pool": "bf16", "new": "64", "ctx": "100000", "hq": 32, "hkv": 8,
         "d": 128, "page": 128, "window": 0, "sink": 0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pieces(rng, n, total):
    """n lengths that sum to total, some of them 0."""
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [y - x for x, y in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "prompt", "prompt"])
    c = {"op": op, "pool": rng.choice(["bf16", "e4m3"]), "hkv": rng.choice([1, 2, 3, 4, 8]), "d": rng.choice([64, 128]),
         "page": rng.choice([16, 32, 64, 128])}
    grp = rng.choice([1, 2, 3, 4, 5, 8])
    windowed = rng.random() < 0.35
    look = {"window": _log_uniform(rng, 1, 4096) if windowed else 0, "sink": rng.choice([0, 1, 4, 33]) if windowed else 0}
    if op == "write":
        n = rng.choice([1, 1, 2, 5, 8])
        return {**c, "src": rng.choice(["bf16", "bf16", "f32"]),
                "new": ",".join(map(str, _pieces(rng, n, _log_uniform(rng, 1, 32768)))),
                "ctx": ",".join(str(rng.randint(0, 2000)) for _ in range(n))}
    if op == "decode":
        cap = c["page"] * max(1, _log_uniform(rng, 64, 32768) // c["page"])
        t = min(rng.choice([1, 1, 1, 2, 3, 5]), cap)
        return {**c, "b": _log_uniform(rng, 1, 12), "t": t, "hq": c["hkv"] * grp, "cap": cap,
                "ctx": rng.randint(max(t, cap // 2), cap), "ragged": rng.random() < 0.7, **look}
    n = rng.choice([1, 1, 2, 3, 5])
    total = _log_uniform(rng, 16, 4096)
    far = _log_uniform(rng, 16, 12288 // n)
    return {**c, "new": ",".join(map(str, _pieces(rng, n, total))),
            "ctx": ",".join(str(rng.randint(0, far)) for _ in range(n)), "hq": min(c["hkv"] * grp, 32 // c["hkv"] * c["hkv"]),
            **look}


def _numbers(text):
    return [int(x) for x in text.split(",")]


def _lengths(case):
    """(new tokens, slots in use with them) of every sequence."""
    if case["op"] == "decode":
        b, t, ctx = case["b"], case["t"], case["ctx"]
        # ragged batches go down to a quarter
        cut = [(ctx * 3 * i) // (4 * max(1, b - 1)) if case["ragged"] else 0 for i in range(b)]
        return [t] * b, [max(t, ctx - x) for x in cut]
    new = _numbers(case["new"])
    return new, [x + y for x, y in zip(new, _numbers(case["ctx"]))]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    hkv, d, page = case["hkv"], case["d"], case["page"]
    new, lens = _lengths(case)
    b = len(new)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # a table as wide as the longest sequence may get; pages lie in the pool in no order
    width = case["cap"] // page if case["op"] == "decode" else max(1, max(-(-x // page) for x in lens))
    held = [-(-x // page) for x in lens]
    n = max(1, sum(held))
    order = torch.randperm(n, generator=g, device=dev).int()
    table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    at = torch.arange(width, device=dev)
    there = at < torch.tensor(held, device=dev)[:, None]
    table[there] = order[:sum(held)]

    s = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "start": torch.tensor([x - y for x, y in zip(lens, new)], dtype=torch.int32, device=dev)}
    shape = (n, hkv, page, d)
    if case["pool"] == "bf16":
        s["pool"] = [normal(*shape).to(torch.bfloat16) for _ in range(2)]
    else:       # bell-shaped rows whose largest value is around three
        s["pool"] = [normal(*shape).mul_(110.0).clamp_(-448.0, 448.0).to(_CODE) for _ in range(2)]
        s["pool"] += [torch.randint(119, 122, shape[:3], generator=g, device=dev, dtype=torch.uint8) for _ in range(2)]

    src = torch.float32 if case.get("src") == "f32" else torch.bfloat16
    packed = case["op"] == "prompt" or (case["op"] == "write" and len(set(new)) > 1)
    rows = (sum(new),) if packed else (b, new[0])
    s["k"], s["v"] = normal(*rows, hkv, d).to(src), normal(*rows, hkv, d).to(src)
    if packed:
        cu = torch.zeros(b + 1, dtype=torch.int32, device=dev)
        cu[1:] = torch.tensor(new, device=dev).cumsum(0)
        s["cu"] = cu
    if case["op"] != "write":
        s["q"] = normal(*rows, case["hq"], d).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    _append_plain(state, case)
    fresh = _read_plain(state, case)
    if case["op"] == "write":
        return fresh
    return (*_attend_plain(state, case), *fresh)


def _own(s, case):
    from sequence_exact_attention_gb300 import binding as ra

    cache, new = ra.PagedCache(*s["pool"]), _lengths(case)[0]
    if "cu" in s:
        ra.paged_append_varlen(cache, s["table"], s["k"], s["v"], s["cu"], s["start"])
    else:
        ra.paged_append(cache, s["table"], s["k"], s["v"], s["start"])
    fresh = ra.paged_read(cache, s["table"], s["start"], max(new))
    if case["op"] == "write":
        return fresh
    look = {"window": case["window"], "n_sink": case["sink"]}
    if case["op"] == "decode":
        return (*ra.paged_attn(s["q"], cache, s["table"], s["lens"], **look), *fresh)
    return (*ra.paged_attn_varlen(s["q"], cache, s["table"], s["lens"], s["cu"], max(new), **look), *fresh)


# ---- plain forms

def _power(byte):
    """2^(byte - 127) as float32."""
    return (byte.int() << 23).view(torch.float32)


def _append_plain(s, case):
    """Writes the new tokens to the pool."""
    new, _ = _lengths(case)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    dev = s["table"].device
    count = torch.tensor(new, device=dev)
    seq = torch.arange(len(new), device=dev).repeat_interleave(count, output_size=sum(new))
    first = count.cumsum(0) - count
    slot = s["start"].long()[seq] + torch.arange(sum(new), device=dev) - first[seq]
    at, row = s["table"].long()[seq, slot // page], slot % page
    for i, name in enumerate("kv"):
        x = s[name].reshape(-1, hkv, d)
        if case["pool"] == "bf16":
            s["pool"][i][at, :, row] = x.to(torch.bfloat16)
            continue
        x = x.float()
        m, e = torch.frexp(x.abs().amax(-1))              # m in [1/2, 1)
        e = torch.where(m > 0, e - 9 + (m > 0.875), -117).clamp_(min=-117)
        code = (x * _power(127 - e)[..., None]).to(_CODE)
        s["pool"][i].view(torch.uint8)[at, :, row] = code.view(torch.uint8)
        s["pool"][2 + i][at, :, row] = (e + 127).to(torch.uint8)


def _slots(s, case, slot):
    """Keys and values [b, t, hkv, d] float32 of slots [b, t], and which of them are there."""
    page, width = case["page"], s["table"].shape[1]
    p = slot // page
    at = s["table"].long().gather(1, p.clamp(max=width - 1))
    there = (p < width) & (at >= 0)
    at, row = at.clamp(min=0), slot % page
    got = []
    for i in range(2):
        pool = s["pool"][i]
        if case["pool"] == "bf16":
            x = pool[at, :, row].float()
        else:
            x = pool.view(torch.uint8)[at, :, row].view(_CODE).float()
            x.mul_(_power(s["pool"][2 + i][at, :, row])[..., None])
        got.append(x)
    return got[0], got[1], there


def _read_plain(s, case):
    t = max(_lengths(case)[0])
    slot = s["start"].long()[:, None] + torch.arange(t, device=s["table"].device)
    k, v, there = _slots(s, case, slot)
    return tuple(x.mul_(there[..., None, None]).to(torch.bfloat16) for x in (k, v))


def _attend_plain(s, case):
    new, lens = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    b, t, grp, dev = len(new), max(new), hq // hkv, s["table"].device
    n = max(lens)
    count = torch.tensor(new, device=dev)
    tok = torch.arange(t, device=dev)
    pad = tok < count[:, None]                                                     # [b, t]
    if "cu" in s:       # packed rows to a padded batch
        row = (s["cu"][:-1].long()[:, None] + tok).clamp(max=sum(new) - 1)
        q = s["q"][row].float()
    else:
        q = s["q"].float()
    q = q.view(b, t, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * grp, d)
    j = torch.arange(n, device=dev)
    k, v, there = _slots(s, case, j.expand(b, n))
    at = (s["lens"].long() - count)[:, None, None] + tok[:, None]                  # [b, t, 1]
    see = (j <= at) & there[:, None]
    if case["window"]:
        see = see & ((j > at - case["window"]) | (j < case["sink"]))
    z = (q @ k.permute(0, 2, 3, 1)).view(b, hkv, t, grp, n).mul_(1.0 / math.sqrt(d))
    z.masked_fill_(~see[:, None, :, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total.clamp(min=1.0))        # a row that sees a slot sums to 1 or more
    o = (p.view(b, hkv, t * grp, n) @ v.permute(0, 2, 1, 3)).view(b, hkv, t, grp, d)
    out = o.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(torch.bfloat16)
    lse = (top + total.log())[..., 0].permute(0, 1, 3, 2).reshape(b, hq, t)
    if "cu" not in s:
        return out, lse
    return out[pad], lse.permute(1, 0, 2)[:, pad].contiguous()


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    new, lens = _lengths(case)
    hkv, d = case["hkv"], case["d"]
    fresh = [[x.reshape(-1, hkv, d)[sum(new[:i]):sum(new[:i + 1])] for i in range(len(new))] for x in (s["k"], s["v"])]
    held = _fresh_exact(s, case, fresh, new, lens)
    if case["op"] == "write":
        return held
    hq, grp = case["hq"], case["hq"] // hkv
    outs, lses = [], []
    for i, (n, length) in enumerate(zip(new, lens)):
        k, v = _rows_exact(s, case, i, 0, length)
        k[length - n:], v[length - n:] = _held(fresh[0][i], case), _held(fresh[1][i], case)
        q = s["q"].reshape(-1, hq, d)[sum(new[:i]):sum(new[:i + 1])].double()
        out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(hq, n, dtype=torch.float64, device="cuda")
        j = torch.arange(length, device="cuda")
        for r in range(0, n, 512):
            p = length - n + torch.arange(r, min(r + 512, n), device="cuda")[:, None]
            hide = j > p
            if case["window"]:
                hide |= (p - j >= case["window"]) & (j >= case["sink"])
            for h in range(hq):
                z = q[r:r + 512, h] @ k[:, h // grp].T * d ** -0.5
                z[hide] = -math.inf
                lse[h, r:r + 512] = torch.logsumexp(z, -1)
                out[r:r + 512, h] = torch.exp(z - lse[h, r:r + 512, None]) @ v[:, h // grp]
        outs.append(out)
        lses.append(lse)
    if case["op"] == "decode":
        return torch.stack(outs), torch.stack(lses), *held
    return torch.cat(outs), torch.cat(lses, 1), *held


def _fresh_exact(s, case, fresh, new, lens):
    """The slots from the new tokens' first on, as far as the longest piece: the new tokens' values, behind them what
    the rest of the last page held before, zeros where no page is."""
    t, page = max(new), case["page"]
    got = [torch.zeros(len(new), t, *fresh[0][0].shape[1:], dtype=torch.float64, device="cuda") for _ in range(2)]
    for i, n in enumerate(new):
        first = lens[i] - n
        last = min(t, -(-lens[i] // page) * page - first)
        for x, old, y in zip(got, _rows_exact(s, case, i, first, first + last), fresh):
            x[i, :last] = old
            x[i, :n] = _held(y[i], case)
    return tuple(got)


def _rows_exact(s, case, i, lo, hi):
    """Keys and values [hi - lo, hkv, d] of sequence i's slots lo to hi, as the pool holds them before the pass."""
    j = torch.arange(lo, hi, device="cuda")
    at = s["table"][i, j // case["page"]].long()
    got = []
    for side in range(2):
        if case["pool"] == "bf16":
            x = s["pool"][side][at, :, j % case["page"]].double()
        else:
            x = s["pool"][side].view(torch.uint8)[at, :, j % case["page"]].view(_CODE).double()
            x *= _power64(s["pool"][2 + side][at, :, j % case["page"]].long() - 127)[..., None]
        got.append(x)
    return got


def _held(x, case):
    """The values that rows x are held as: an e4m3 number has steps of an eighth of its power of two, from 2^-6 on."""
    if case["pool"] == "bf16":
        return x.to(torch.bfloat16).double()
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -120) / 448.0)).clamp(min=-117).long()
    y = x / _power64(e)
    step = _power64(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).long() - 3)
    return torch.round(y / step) * step * _power64(e)


def _power64(e):
    """2^e, exactly."""
    return ((e + 1023) << 52).view(torch.float64)


# ------------------------------------------------------------------ work

def _pairs(new, length, window, sink):
    """(query, slot) pairs of the last `new` of `length` slots, and slots that one of them sees."""
    if not new:
        return 0, 0
    first = length - new + 1                        # slots up to the first new token's
    if not window:
        return new * first + new * (new - 1) // 2, length
    pairs = sum(min(p, window) + min(max(p - window, 0), sink) for p in range(first, length + 1))
    return pairs, min(length, window + new - 1 + sink)


def work(case):
    new, lens = _lengths(case)
    hkv, d = case["hkv"], case["d"]
    row = 2 * d if case["pool"] == "bf16" else d + 1      # bytes of a row as it is held
    total = sum(new)
    src = 4 if case.get("src") == "f32" else 2
    t = max(new)
    back = sum(min(t, -(-x // case["page"]) * case["page"] - (x - n)) for n, x in zip(new, lens))
    # the new tokens in and down, and the values read back
    moved = 2 * hkv * (total * (src * d + row) + back * row + len(new) * t * 2 * d)
    if case["op"] == "write":
        return {"bytes": moved, "flops": 2 * total * hkv * d}
    hq = case["hq"]
    seen = [_pairs(n, x, case["window"], case["sink"]) for n, x in zip(new, lens)]
    io = total * hq * (4 * d + 4)
    return {"bytes": moved + 2 * sum(x[1] for x in seen) * hkv * row + io, "flops": 4 * hq * d * sum(x[0] for x in seen)}
