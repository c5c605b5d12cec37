"""Cases of the cache and attention operators: writing and reading a quantised key/value cache, attention of
drafted tokens over it, and causal attention over packed prompts.

``run`` computes a case in a plain form of elementary torch operations (``own = False``) or by the library's
operators (``own = True``).  ``exact`` has the definitions in 64 bits.

What the operators compute
  cache formats (per token and head, a vector of d values; statistics in 32 bits):
    f16    the values, rounded to fp16
    int8   a = max|x| / 127, code = clamp(rint(x / a), -127, 127) (0 for a zero vector), value = code * a
    q4_0   per 32 values: a = (the signed value of largest magnitude, the first one on ties) / -8,
           code = clamp(round_half_away(x / a) + 8, 0, 15) (8 for a zero block), value = (code - 8) * fp16(a)
  drafted tokens: token i of a sequence sees the sequence's first ctx cached positions, and position ctx + j where
    bit j of its mask is set; out = softmax(scale * q . k) . v, lse = log sum exp(scale * q . k)
  prompts: query i of a sequence of nq queries and nk keys sees the keys j <= i + nk - nq
  A row that sees nothing gives out = 0 and lse = -inf.
"""
import math
import random

import torch

own = False

HEADS = {"32x128": (32, 32, 128),   # 4096 = 32 heads of 128, a key/value head for each
         "64/8x128": (64, 8, 128),  # 8192 = 64 heads of 128 in 8 groups
         "40/8x128": (40, 8, 128),  # 5120 = 40 heads of 128 in 8 groups of 5
         "16/2x64": (16, 2, 64)}    # small heads


# ------------------------------------------------------------------ cases --

def listed():
    kv, tree, prompt = {"op": "kv"}, {"op": "tree"}, {"op": "prompt"}
    return [
        # one decoded token of one sequence goes into the cache, from the fp32 rows of a q|k|v product
        {**kv, "name": "kv int8 one token", "fmt": "int8", "type": "f32", "heads": "64/8x128", "page": 64, "seqs": 1,
         "past": 700, "new": 1, "read": "new", "mix": 1},
        # prompts of several lengths go into small pages
        {**kv, "name": "kv q4_0 prompts", "fmt": "q4_0", "type": "f16", "heads": "40/8x128", "page": 16, "seqs": 5,
         "past": 90, "new": 1500, "read": "new", "mix": 2},
        # a chunk of a prompt is added, and all of the sequences so far read back for its attention
        {**kv, "name": "kv f16 chunk and past", "fmt": "f16", "type": "f16", "heads": "32x128", "page": 32, "seqs": 3,
         "past": 9000, "new": 512, "read": "all", "mix": 3},
        # long prompts of many heads
        {**kv, "name": "kv int8 long prompts", "fmt": "int8", "type": "f32", "heads": "32x128", "page": 128, "seqs": 4,
         "past": 0, "new": 9001, "read": "new", "mix": 4},
        # one token decoded early in a chat: latency counts
        {**tree, "name": "tree int8 one token", "fmt": "int8", "heads": "32x128", "page": 64, "seqs": 1, "past": 511,
         "new": 1, "mix": 5},
        # a tree of 16 drafted tokens, the most that the packed products take at once
        {**tree, "name": "tree int8 16 drafts", "fmt": "int8", "heads": "64/8x128", "page": 64, "seqs": 1, "past": 8000,
         "new": 16, "mix": 6},
        # sequences of different lengths, trees of different sizes, in small pages
        {**tree, "name": "tree q4_0 batch", "fmt": "q4_0", "heads": "40/8x128", "page": 16, "seqs": 12, "past": 20000,
         "new": 9, "mix": 7},
        # two long documents
        {**tree, "name": "tree f16 long", "fmt": "f16", "heads": "64/8x128", "page": 256, "seqs": 2, "past": 131000,
         "new": 5, "mix": 8},
        # a handful of short prompts: latency counts
        {**prompt, "name": "prompt short", "type": "f16", "heads": "32x128", "seqs": 8, "past": 0, "new": 64, "mix": 9},
        # prompts of different lengths packed together
        {**prompt, "name": "prompt packed bf16", "type": "bf16", "heads": "64/8x128", "seqs": 4, "past": 0,
         "new": 4000, "mix": 10},
        # chunks of prompts after a past that was read back from the cache
        {**prompt, "name": "prompt chunk", "type": "f16", "heads": "40/8x128", "seqs": 2, "past": 6000, "new": 300,
         "mix": 11},
        # one long prompt
        {**prompt, "name": "prompt long", "type": "f16", "heads": "64/8x128", "seqs": 1, "past": 0, "new": 8192,
         "mix": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    c = {"op": rng.choice(["kv", "tree", "prompt"]), "heads": rng.choice(sorted(HEADS)), "mix": rng.randrange(1, 1 << 20)}
    hq, hkv, d = HEADS[c["heads"]]
    if c["op"] == "prompt":
        # scores of the padded plain form: seqs * hq * new * (new + past), at most those of one prompt of 8192
        c |= {"type": rng.choice(["f16", "bf16"]), "seqs": _log(rng, 1, 24), "new": _log(rng, 1, 8192),
              "past": rng.choice([0, _log(rng, 1, 8192)])}
        while c["seqs"] * hq * c["new"] * (c["new"] + c["past"]) > 64 * 8192 * 4096:
            k = max(("seqs", "new", "past"), key=lambda n: c[n] * (200 if n == "seqs" else 1))
            c[k] = c[k] // 2
        return c
    c |= {"fmt": rng.choice(["f16", "int8", "q4_0"]), "page": rng.choice([16, 32, 64, 128, 256]), "seqs": _log(rng, 1, 48)}
    if c["op"] == "kv":
        c |= {"type": rng.choice(["f32", "f16", "bf16"]), "new": _log(rng, 1, 9000), "past": _log(rng, 1, 9000) - 1,
              "read": rng.choice(["new", "all"])}
        most = 4 * 9001 * 32 * 128
    else:
        c |= {"new": _log(rng, 1, 16), "past": _log(rng, 1, 131000) - 1}
        most = 2 * 131000 * 8 * 128
    while c["seqs"] * (c["past"] + c["new"]) * hkv * d > most:
        k = max(("seqs", "new", "past"), key=lambda n: c[n] * (200 if n == "seqs" else 1))
        c[k] = c[k] // 2
    return c


def _lens(case):
    """(cached tokens before, new tokens) of each sequence: the first has the most; among several, one is short."""
    r = random.Random(case["mix"])
    n = case["seqs"]
    past, new = [case["past"]], [case["new"]]
    for i in range(1, n):
        past.append(r.randint(0, case["past"]) if i % 5 else r.randint(0, min(20, case["past"])))
        new.append(r.randint(1, case["new"]) if i % 3 else min(case["new"], r.randint(1, 3)))
    return past, new


def _value_bytes(fmt, d):
    return {"f16": 2 * d, "int8": d + 4, "q4_0": d // 32 * 18}[fmt]


def work(case):
    hq, hkv, d = HEADS[case["heads"]]
    past, new = _lens(case)
    if case["op"] == "kv":
        n = sum(new)
        rows = n if case["read"] == "new" else n + sum(past)
        size = {"f32": 4, "f16": 2, "bf16": 2}[case["type"]]
        one = _value_bytes(case["fmt"], d)
        # new rows read, their codes written; codes read and fp16 rows written of what is read back
        return {"bytes": 2 * hkv * (n * (size * d + one) + rows * (one + 2 * d)) + 8 * n, "flops": 8 * hkv * d * (n + rows)}
    if case["op"] == "tree":
        one = _value_bytes(case["fmt"], d)
        seen = [_bits(m) for m in _masks(case)]
        at, pairs = 0, 0
        for p, n in zip(past, new):
            pairs += sum(p + s for s in seen[at:at + n])
            at += n
        cached = sum(past) + sum(new)
        return {"bytes": 2 * hkv * cached * one + sum(new) * hq * (4 * d + 4) + 8 * sum(new) + 4 * (cached // case["page"]),
                "flops": 4 * d * hq * pairs}
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, new))
    return {"bytes": sum(new) * hq * (4 * d + 4) + 4 * d * hkv * (sum(new) + sum(past)), "flops": 4 * d * hq * pairs}


def _bits(m):
    return bin(m).count("1")


def _masks(case):
    """The drafted tokens' masks: a random tree for each sequence; token i sees its ancestors and itself."""
    r = random.Random(case["mix"] + 1)
    got = []
    for n in _lens(case)[1]:
        mine = []
        for i in range(n):
            up = r.randrange(max(0, i - 4), i) if i else None
            mine.append((mine[up] if i else 0) | 1 << i)
        got += mine
    return got


# ----------------------------------------------------------------- inputs --

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _stack(case, seed, rows, kind, tag):
    """Rows of a stacked q|k|v product: values of N(0, 1), some channels of k larger, as such products have them."""
    hq, hkv, d = HEADS[case["heads"]]
    g = torch.Generator(device="cuda").manual_seed(seed * 16 + tag)
    x = torch.randn(rows, (hq + 2 * hkv) * d, generator=g, device="cuda", dtype=torch.float32)
    big = torch.exp(0.5 * torch.randn(hkv * d, generator=g, device="cuda", dtype=torch.float32))
    x[:, hq * d:(hq + hkv) * d] *= big
    x = x.to(kind)
    cut = lambda at, h: x[:, at * d:(at + h) * d].unflatten(1, (h, d))  # noqa: E731
    return cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv)


def _pairs(case, seed, rows, kind, tag):
    """k and v rows alone, as _stack has them."""
    hq, hkv, d = HEADS[case["heads"]]
    g = torch.Generator(device="cuda").manual_seed(seed * 16 + tag)
    big = torch.exp(0.5 * torch.randn(hkv * d, generator=g, device="cuda", dtype=torch.float32)).view(hkv, d)
    k = torch.randn(rows, hkv, d, generator=g, device="cuda", dtype=torch.float32) * big
    v = torch.randn(rows, hkv, d, generator=g, device="cuda", dtype=torch.float32)
    return k.to(kind), v.to(kind)


def _sums(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _slots(table, page, lo, n):
    """Slots (page * page size + place) of the positions lo .. lo + n of every sequence, packed."""
    n, lo = torch.as_tensor(n, device="cuda"), torch.as_tensor(lo, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    start = torch.cumsum(n, 0) - n
    pos = torch.arange(len(seq), device="cuda") - start[seq] + lo[seq]
    return table[seq, pos // page].long() * page + pos % page


def _table(case, seed):
    past, new = _lens(case)
    page, most = case["page"], -(-max(p + n for p, n in zip(past, new)) // case["page"])
    n_pages = sum(-(-(p + n) // page) for p, n in zip(past, new)) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, at = torch.full((len(past), most), -1, dtype=torch.int32), 0
    for i, (p, n) in enumerate(zip(past, new)):
        m = -(-(p + n) // page)
        table[i, :m] = order[at:at + m]
        at += m
    return table.cuda(), n_pages


def _plain_cache(case, n_pages):
    hq, hkv, d = HEADS[case["heads"]]
    n = n_pages * case["page"]
    if case["fmt"] == "f16":
        return {s: torch.zeros(n, hkv, d, dtype=torch.float16, device="cuda") for s in ("k", "v")}
    groups = 1 if case["fmt"] == "int8" else d // 32
    kind = torch.float32 if case["fmt"] == "int8" else torch.float16
    c = {s: torch.zeros(n, hkv, d, dtype=torch.int8, device="cuda") for s in ("k", "v")}
    return c | {s + "_scale": torch.zeros(n, hkv, groups, dtype=kind, device="cuda") for s in ("k", "v")}


def prepare(case, seed):
    hq, hkv, d = HEADS[case["heads"]]
    past, new = _lens(case)
    st = {"case": case, "past": past, "new": new, "cu_new": _sums(new), "scale": 1 / math.sqrt(d)}
    if case["op"] == "prompt":
        kind = TYPES[case["type"]]
        if case["past"] == 0:
            st["q"], st["k"], st["v"] = _stack(case, seed, sum(new), kind, 1)
        else:
            st["q"] = _stack(case, seed, sum(new), kind, 1)[0]
            st["k"], st["v"] = _pairs(case, seed, sum(new) + sum(past), kind, 2)
        st["cu_all"] = _sums([p + n for p, n in zip(past, new)])
        if own:
            from bit_weight_only_gb300 import qgemv
            st["ws"] = qgemv.AttnWorkspace(len(new), hq, d)
        else:
            st["pad"] = _padding(past, new)
        return st
    # a cache: the past is in it; for a tree the drafted tokens too
    table, n_pages = _table(case, seed)
    st |= {"table": table, "n_pages": n_pages}
    zero = [0] * len(past)
    every = [p + n for p, n in zip(past, new)]
    fill = past if case["op"] == "kv" else every
    k, v = _pairs(case, seed, sum(fill), torch.float16, 3)
    slots = _slots(table, case["page"], zero, fill)
    if own:
        from bit_weight_only_gb300 import qgemv
        st["cache"] = qgemv.KVCache(case["fmt"], n_pages, case["page"], hkv, d)
        st["cache"].write(k, v, slots)
    else:
        st["cache"] = _plain_cache(case, n_pages)
        _plain_write(case["fmt"], st["cache"], k, v, slots)
    if case["op"] == "kv":
        _, st["k"], st["v"] = _stack(case, seed, sum(new), TYPES[case["type"]], 4)
        st["slots"] = _slots(table, case["page"], past, new)
        starts, n = (past, new) if case["read"] == "new" else (zero, every)
        st |= {"starts": torch.tensor(starts, dtype=torch.int32, device="cuda"), "cu_read": _sums(n), "n_read": sum(n)}
        return st
    st["q"] = _stack(case, seed, sum(new), torch.float16, 5)[0]
    st["ctx"] = torch.tensor(past, dtype=torch.int32, device="cuda")
    st["masks"] = torch.tensor([m - (1 << 64 if m >> 63 else 0) for m in _masks(case)], dtype=torch.int64, device="cuda")
    if own:
        st["ws"] = qgemv.AttnWorkspace(len(new), hq, d)
    else:
        st["pad"] = _padding(past, new)
    return st


def _padding(past, new):
    """Places of packed rows in a padded batch, and back: (rows of new tokens, rows of all tokens)."""
    def of(n):
        n = torch.tensor(n, device="cuda")
        at = torch.arange(int(n.max()), device="cuda")
        start = torch.cumsum(n, 0) - n
        there = at[None] < n[:, None]
        return {"rows": torch.where(there, start[:, None] + at[None], 0), "there": there}
    return of(new), of([p + n for p, n in zip(past, new)])


# ------------------------------------------------------------- plain form --

def _plain_codes(fmt, x):
    x = x.float()
    if fmt == "int8":
        a = x.abs().amax(-1, keepdim=True)
        a = a / torch.full_like(a, 127)  # a division (by a plain number torch multiplies by its reciprocal)
        q = torch.where(a > 0, torch.clamp(torch.round(x / a), -127, 127), torch.zeros_like(x))
        return q.to(torch.int8), a
    b = x.unflatten(-1, (-1, 32))
    m = b.abs()
    a = torch.gather(b, -1, m.argmax(-1, keepdim=True)) / -8
    r = b / a
    r = torch.sign(r) * torch.floor(r.abs() + 0.5)  # half away from zero
    q = torch.where(a != 0, torch.clamp(r + 8, 0, 15) - 8, torch.zeros_like(b))
    return q.to(torch.int8).flatten(-2), a.squeeze(-1).to(torch.float16)


def _plain_write(fmt, cache, k, v, slots):
    for s, x in (("k", k), ("v", v)):
        if fmt == "f16":
            cache[s][slots] = x.to(torch.float16)
        else:
            cache[s][slots], cache[s + "_scale"][slots] = _plain_codes(fmt, x)


def _plain_values(fmt, cache, s, slots):
    x = cache[s][slots].float()
    if fmt == "f16":
        return x
    a = cache[s + "_scale"][slots].float()
    return (x.unflatten(-1, (a.shape[-1], -1)) * a[..., None]).flatten(-2)


def _plain_softmax(s, see, v):
    """(out, lse) of scores s [..., rows, keys], of which `see` count, and values v [..., keys, d]."""
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    s -= top
    p = s.exp_()
    n = p.sum(-1, keepdim=True)
    out = p @ v / torch.where(n > 0, n, torch.ones_like(n))
    return out, (top + n.log()).squeeze(-1)


def _plain_attention(q, k, v, see, scale):
    """q [b, rows, hq, d], k and v [b, keys, hkv, d], see [b, rows, keys] -> out [b, rows, hq, d], lse [b, rows, hq]"""
    b, rows, hq, d = q.shape
    hkv = k.shape[2]
    q = q.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)      # b, hkv, g * rows, d
    k, v = k.permute(0, 2, 3, 1), v.permute(0, 2, 1, 3)
    s = (q @ k).mul_(scale).unflatten(2, (hq // hkv, rows))                          # b, hkv, g, rows, keys
    out, lse = _plain_softmax(s, see[:, None, None], v[:, :, None])
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)


def _plain_run(st):
    case = st["case"]
    if case["op"] == "kv":
        _plain_write(case["fmt"], st["cache"], st["k"], st["v"], st["slots"])
        n = st["cu_read"][1:] - st["cu_read"][:-1]
        slots = _slots(st["table"], case["page"], st["starts"], n)
        k, v = (_plain_values(case["fmt"], st["cache"], s, slots).to(torch.float16) for s in ("k", "v"))
        return {"k": k, "v": v}
    mine, every = st["pad"]
    past = torch.tensor(st["past"], device="cuda")
    new = st["cu_new"][1:] - st["cu_new"][:-1]
    q = st["q"].float()[mine["rows"]]
    rows, keys = mine["rows"].shape[1], every["rows"].shape[1]
    at = torch.arange(keys, device="cuda")
    if case["op"] == "tree":
        place = at.expand(len(past), keys)
        slots = torch.where(every["there"], st["table"][torch.arange(len(past), device="cuda")[:, None], place // case["page"]].long()
                            * case["page"] + place % case["page"], 0)
        k, v = (_plain_values(case["fmt"], st["cache"], s, slots) for s in ("k", "v"))
        j = at[None] - past[:, None]                                                 # b, keys
        bit = (st["masks"][mine["rows"]][:, :, None] >> j.clamp(0, 63)[:, None]) & 1
        see = (j < 0)[:, None] | ((j < new[:, None])[:, None] & (bit == 1))
        see = see & every["there"][:, None]
    else:
        k, v = st["k"].float()[every["rows"]], st["v"].float()[every["rows"]]
        see = at[None, None] <= (torch.arange(rows, device="cuda")[None] + past[:, None])[:, :, None]
        see = see & every["there"][:, None]
    out, lse = _plain_attention(q, k, v, see, st["scale"])
    return {"out": out[mine["there"]].to(st["q"].dtype), "lse": lse[mine["there"]]}


# -------------------------------------------------------------------- run --

def run(st):
    if not own:
        return _plain_run(st)
    from bit_weight_only_gb300 import qgemv
    case = st["case"]
    if case["op"] == "kv":
        st["cache"].write(st["k"], st["v"], st["slots"])
        k, v = st["cache"].read(st["table"], st["starts"], st["cu_read"], st["n_read"])
        return {"k": k, "v": v}
    if case["op"] == "tree":
        out, lse = st["cache"].attend(st["q"], st["table"], st["ctx"], st["cu_new"], st["masks"], max_ctx=max(st["past"]),
                                      max_new=max(st["new"]), scale=st["scale"], workspace=st["ws"])
    else:
        out, lse = qgemv.attn_prompt(st["q"], st["k"], st["v"], st["cu_new"], st["cu_all"], max_q=max(st["new"]),
                                     scale=st["scale"], workspace=st["ws"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ exact --

def _exact_values(fmt, x):
    """What the cache stands for, in 64 bits; the codes are decided in 32 bits, by definition."""
    if fmt == "f16":
        return x.to(torch.float16).double()
    x = x.to(torch.float32)
    if fmt == "int8":
        a = torch.max(x, -1, keepdim=True).values.maximum(-torch.min(x, -1, keepdim=True).values)
        a = a / torch.tensor([127.0], device=x.device)
        q = torch.where(a == 0, 0.0, (x / a)).round().clamp(-127, 127)
        return q.double() * a.double()
    got = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for lo in range(0, x.shape[-1], 32):
        b = x[..., lo:lo + 32]
        top, low = b.max(-1), b.min(-1)
        peak = torch.where((top.values > -low.values) | ((top.values == -low.values) & (top.indices < low.indices)), top.values, low.values)
        a = (peak / -8)[..., None]
        r = torch.where(a == 0, 0.0, b / a)
        r = torch.trunc(r.double() + torch.where(r < 0, -0.5, 0.5).double())
        got[..., lo:lo + 32] = r.clamp(-8, 7) * a.to(torch.float16).double()
    return got


def _exact_attention(q, k, v, see, scale):
    """q [rows, hq, d], k, v [keys, hkv, d], see [rows, keys]; a head at a time."""
    rows, hq, d = q.shape
    per = hq // k.shape[1]
    out = torch.zeros(rows, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device="cuda")
    some = see.any(1)
    for h in range(hq):
        s = (q[:, h] @ k[:, h // per].T) * scale
        s[~see] = -math.inf
        lse[:, h] = torch.logsumexp(s, 1)
        p = torch.softmax(s, 1)
        p[~some] = 0
        out[:, h] = p @ v[:, h // per]
    return out, lse


def exact(case, seed):
    hq, hkv, d = HEADS[case["heads"]]
    past, new = _lens(case)
    if work(case)["flops"] > 1.5e12:
        return None  # 64-bit products of this size take too long
    if case["op"] == "kv":
        _, k, v = _stack(case, seed, sum(new), TYPES[case["type"]], 4)
        k, v = _exact_values(case["fmt"], k), _exact_values(case["fmt"], v)
        if case["read"] == "new":
            return {"k": k, "v": v}
        k0, v0 = (_exact_values(case["fmt"], x) for x in _pairs(case, seed, sum(past), torch.float16, 3))
        ks, vs, a, b = [], [], 0, 0
        for p, n in zip(past, new):
            ks += [k0[a:a + p], k[b:b + n]]
            vs += [v0[a:a + p], v[b:b + n]]
            a, b = a + p, b + n
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    outs, lses, a, b = [], [], 0, 0
    if case["op"] == "tree":
        q = _stack(case, seed, sum(new), torch.float16, 5)[0].double()
        k, v = _pairs(case, seed, sum(past) + sum(new), torch.float16, 3)
        masks = _masks(case)
    elif case["past"] == 0:
        q, k, v = (x.double() for x in _stack(case, seed, sum(new), TYPES[case["type"]], 1))
    else:
        q = _stack(case, seed, sum(new), TYPES[case["type"]], 1)[0].double()
        k, v = (x.double() for x in _pairs(case, seed, sum(new) + sum(past), TYPES[case["type"]], 2))
    for p, n in zip(past, new):
        if case["op"] == "tree":
            see = torch.ones(n, p + n, dtype=torch.bool)
            see[:, p:] = torch.tensor([[bool(m >> j & 1) for j in range(n)] for m in masks[b:b + n]])
            kk, vv = (_exact_values(case["fmt"], x[a:a + p + n]) for x in (k, v))
        else:
            see = torch.ones(n, p + n, dtype=torch.bool).tril(p)
            kk, vv = k[a:a + p + n], v[a:a + p + n]
        o, l = _exact_attention(q[b:b + n], kk, vv, see.cuda(), scale=1 / math.sqrt(d))
        outs.append(o)
        lses.append(l)
        a, b = a + p + n, b + n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
