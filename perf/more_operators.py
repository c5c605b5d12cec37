"""Cases of the operators around the paged cache: rotary positions of several axes on the way into it, beam search's selection,
forking and compacting of its pages, and attention over the pages that a cheap score selects.

``run`` computes a case in a plain form of elementary torch operations (``own = False``) or by the library's operators
(``own = True``).  ``exact`` has the definitions in 64 bits.

What the operators compute
  rotary positions: pair j of a head vector belongs to axis(j) of its token's position; (a, b) -> (a cos - b sin, a sin + b cos)
    with the angle position[axis(j)] * base^(-j / pairs); pairs are (j, j + pairs) ("halves") or (2j, 2j + 1) ("neighbours");
    values behind the pairs stay.  Rotated q is returned, rotated k goes into a cache with v.
  selection: of a sequence's candidates (beam b, token t), score[b] + logits[b][t] - log sum exp logits[b], the `width` largest;
    ties go to the lower beam, then the lower token.  A beam whose score or log sum is not finite has none; places without a
    candidate are (-inf, -1, -1).
  forking: row r of the new page table is the old row parents[r]; pages count their rows; the page that a row has filled in
    part is its first child's, the others get a free page each (the lowest, in the rows' order) and a copy of its tokens.
  compacting: the pages in use from number `used` on move, in order, to the free ones below; tables and counts follow.
  selected attention: a whole page before the context's end has a summary for each key/value head, its largest and smallest key
    values per channel in codes, scale = max / 127; the queries' positive and negative parts, summed over a head's queries, are
    in codes too; score = (sum of the codes' products) * the page's scale.  The n_select pages of highest score (ties: the
    earlier) and all positions from the last whole page on are attended, as in perf/operators.py.
"""
import math
import random

import torch

own = False

HEADS = {"32x128": (32, 32, 128),   # 4096 = 32 heads of 128, a key/value head for each
         "64/8x128": (64, 8, 128),  # 8192 = 64 heads of 128 in 8 groups
         "40/8x128": (40, 8, 128),  # 5120 = 40 heads of 128 in 8 groups of 5
         "16/2x64": (16, 2, 64)}    # small heads
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DRAFTS = 64                         # drafted tokens of a sequence, at most


# ------------------------------------------------------------------ cases --

def listed():
    rope, beam, fork, compact, sparse = ({"op": o} for o in ("rope", "beam", "fork", "compact", "sparse"))
    return [
        # one decoded token's q and k, from the fp32 rows of a q|k|v product: latency counts
        {**rope, "name": "rotate one token", "heads": "40/8x128", "type": "f32", "axes": 1, "pairs": "halves", "into": "rows",
         "page": 16, "seqs": 1, "past": 900000, "new": 1, "mix": 1},
        # prompts of text and images (time, height, width), a part of each head rotated, into an INT8 cache and back for attention
        {**rope, "name": "rotate prompts int8", "heads": "64/8x128", "type": "f32", "axes": 3, "pairs": "halves", "into": "int8",
         "page": 64, "seqs": 5, "past": 3000, "new": 1111, "mix": 2},
        # long prompts of many heads
        {**rope, "name": "rotate long f16", "heads": "32x128", "type": "bf16", "axes": 3, "pairs": "neighbours", "into": "f16",
         "page": 128, "seqs": 3, "past": 0, "new": 9001, "mix": 3},
        # one sequence's beams after the 32000-row LM head: latency counts
        {**beam, "name": "select one sequence", "type": "f32", "seqs": 1, "beams": 4, "vocab": 32000, "width": 8, "mix": 4},
        # a batch with an odd vocabulary in 16 bits, where many logits are equal
        {**beam, "name": "select bf16 odd", "type": "bf16", "seqs": 9, "beams": 5, "vocab": 50021, "width": 10, "mix": 5},
        # many sequences, a large vocabulary
        {**beam, "name": "select batch", "type": "f32", "seqs": 64, "beams": 8, "vocab": 128000, "width": 16, "mix": 6},
        # the beams of a short chat change their order: latency counts
        {**fork, "name": "fork 4 beams", "fmt": "int8", "heads": "32x128", "page": 16, "seqs": 1, "beams": 4, "past": 700, "mix": 7},
        # many beams of long sequences in large pages
        {**fork, "name": "fork 16 x 8 beams", "fmt": "f16", "heads": "64/8x128", "page": 256, "seqs": 16, "beams": 8,
         "past": 5000, "mix": 8},
        # a cache full of holes is packed
        {**compact, "name": "compact q4_0", "fmt": "q4_0", "heads": "40/8x128", "page": 64, "pages": 9001, "seqs": 48,
         "past": 12000, "mix": 9},
        # a long prompt's pages get their summaries, then the first token
        {**sparse, "name": "sparse first token", "fmt": "f16", "heads": "32x128", "page": 32, "seqs": 1, "past": 8000, "new": 1,
         "select": 24, "fresh": "all", "mix": 10},
        # one token of a very long document
        {**sparse, "name": "sparse long int8", "fmt": "int8", "heads": "64/8x128", "page": 16, "seqs": 1, "past": 131000, "new": 1,
         "select": 256, "fresh": "last", "mix": 11},
        # drafted tokens of sequences of different lengths
        {**sparse, "name": "sparse batch q4_0", "fmt": "q4_0", "heads": "40/8x128", "page": 64, "seqs": 12, "past": 60000, "new": 4,
         "select": 48, "fresh": "last", "mix": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    c = {"op": rng.choice(["rope", "beam", "fork", "compact", "sparse"]), "mix": rng.randrange(1, 1 << 20)}
    if c["op"] == "beam":
        c |= {"type": rng.choice(["f32", "f16", "bf16"]), "seqs": _log(rng, 1, 64), "beams": _log(rng, 1, 16),
              "vocab": _log(rng, 1000, 128000)}
        c["width"] = c["beams"] * rng.choice([1, 2])
        while c["seqs"] * c["beams"] * c["vocab"] > 64 * 8 * 128000:
            c["seqs"] //= 2
        return c
    c |= {"heads": rng.choice(sorted(HEADS)), "page": rng.choice([16, 32, 64, 128, 256]), "seqs": _log(rng, 1, 48)}
    hq, hkv, d = HEADS[c["heads"]]
    if c["op"] == "rope":
        c |= {"type": rng.choice(["f32", "f16", "bf16"]), "axes": rng.choice([1, 2, 3]), "new": _log(rng, 1, 9000),
              "pairs": rng.choice(["halves", "neighbours"]), "into": rng.choice(["rows", "f16", "int8"]),
              "past": rng.choice([0, _log(rng, 1, 100000)])}
        cost, most = (lambda: c["seqs"] * c["new"] * (hq + 2 * hkv) * d), 3 * 9001 * 96 * 128
        shrink = ("seqs", "new")
    elif c["op"] == "fork":
        c |= {"fmt": rng.choice(["f16", "int8", "q4_0"]), "beams": _log(rng, 1, 16), "past": _log(rng, 1, 20000)}
        cost, most = (lambda: c["seqs"] * (c["past"] * (c["beams"] + 1) // 2 + c["beams"] * c["page"]) * hkv * d), 16 * 24548 * 8 * 128
        shrink = ("seqs", "past")
    elif c["op"] == "compact":
        c |= {"fmt": rng.choice(["f16", "int8", "q4_0"]), "past": _log(rng, 1, 20000)}
        c["pages"] = 0
        cost, most = (lambda: c["seqs"] * c["past"] * hkv * d * (4 if c["fmt"] == "f16" else 2)), 48 * 12000 * 8 * 128
        shrink = ("seqs", "past")
    else:
        c |= {"fmt": rng.choice(["f16", "int8", "q4_0"]), "new": _log(rng, 1, 8), "past": _log(rng, 100, 131000),
              "select": _log(rng, 1, 300), "fresh": rng.choice(["all", "last", "last"])}
        cost, most = (lambda: c["seqs"] * c["past"] * hkv * d), 12 * 60000 * 8 * 128
        shrink = ("seqs", "past")
    while cost() > most:
        k = max(shrink, key=lambda n: c[n] * (200 if n == "seqs" else 1))
        c[k] //= 2
    if c["op"] == "compact":
        c["pages"] = int(_pages_of(c) * rng.uniform(1.3, 2.0)) + 2
    if c["op"] == "sparse":  # the plain form's keys of the selected pages
        while c["seqs"] * hkv * c["select"] * c["page"] * d > 12 * 8 * 3100 * 128:
            c["select"] = max(1, c["select"] // 2)
            if c["select"] == 1:
                break
    return c


def _lens(case):
    """(cached tokens before, new tokens) of each sequence: the first has the most; among several, one is short."""
    r = random.Random(case["mix"])
    past, new = [case["past"]], [case.get("new", 0)]
    for i in range(1, case["seqs"]):
        past.append(r.randint(0, case["past"]) if i % 5 else r.randint(0, min(20, case["past"])))
        new.append((r.randint(1, case["new"]) if i % 3 else min(case["new"], r.randint(1, 3))) if "new" in case else 0)
    return past, new


def _pages_of(case):
    return sum(-(-p // case["page"]) for p in _lens(case)[0])


def _token_bytes(fmt, d):
    """Of one token and head, K and V together."""
    return 2 * {"f16": 2 * d, "int8": d + 4, "q4_0": d // 32 * 18}[fmt]


def _parents(case):
    """A step of beam search: within a sequence some beams go on as several, some as none."""
    r, n = random.Random(case["mix"] + 2), case["beams"]
    got = []
    for s in range(case["seqs"]):
        mine = [min(r.randrange(n), r.randrange(n)) for _ in range(n)]
        got += [s * n + b for b in mine]
    return got


def work(case):
    if case["op"] == "beam":
        rows = case["seqs"] * case["beams"]
        size = {"f32": 4, "f16": 2, "bf16": 2}[case["type"]]
        return {"bytes": rows * (case["vocab"] * size + 4) + case["seqs"] * case["width"] * 12, "flops": 4 * rows * case["vocab"]}
    hq, hkv, d = HEADS[case["heads"]]
    past, new = _lens(case)
    page = case["page"]
    if case["op"] == "rope":
        n = sum(new)
        size = {"f32": 4, "f16": 2, "bf16": 2}[case["type"]]
        if case["into"] == "rows":
            return {"bytes": n * ((hq + hkv) * d * (size + 2) + 4 * case["axes"]), "flops": 4 * n * (hq + hkv) * d}
        one = _token_bytes(case["into"], d)
        # rows read, q and codes written; codes read and fp16 rows written of what is read back
        return {"bytes": n * ((hq + 2 * hkv) * d * size + hq * d * 2 + hkv * (2 * one + 4 * d) + 8 + 4 * case["axes"]),
                "flops": n * (hq + 2 * hkv) * d * 4}
    if case["op"] == "fork":
        parents = _parents(case)
        entries = case["beams"] * _pages_of(case)
        copied = sum((past[b // case["beams"]] % page) for i, b in enumerate(parents) if b in parents[:i])
        # the table and its new form; counts of the pages that change; tokens of the copied pages
        return {"bytes": 8 * entries + 8 * entries // 2 + 2 * copied * hkv * _token_bytes(case["fmt"], d), "flops": entries}
    if case["op"] == "compact":
        used = _pages_of(case)
        moved = used * (case["pages"] - used) // case["pages"]  # of pages in random places
        return {"bytes": 8 * case["pages"] + 8 * used + 2 * moved * page * hkv * _token_bytes(case["fmt"], d), "flops": case["pages"]}
    one = _token_bytes(case["fmt"], d)
    whole = [p // page for p in past]
    seen = [min(w, case["select"]) * page + p % page for w, p in zip(whole, past)]
    fresh = sum(whole) if case["fresh"] == "all" else sum(w > 0 for w in whole)
    pairs = sum(n * s + n * (n + 1) // 2 for s, n in zip(seen, new))
    return {"bytes": hkv * (fresh * (page * one // 2 + 2 * d + 4) + sum(whole) * (2 * d + 4) + (sum(seen) + sum(new)) * one)
            + sum(new) * hq * (4 * d + 4) + 4 * sum(whole) + 4 * hkv * sum(min(w, case["select"]) for w in whole),
            "flops": 4 * d * hq * pairs + 4 * d * hkv * sum(whole)}


# ----------------------------------------------------------------- inputs --

def _gen(seed, tag):
    return torch.Generator(device="cuda").manual_seed(seed * 16 + tag)


def _stack(case, seed, rows, kind, tag):
    """Rows of a stacked q|k|v product: values of N(0, 1), some channels of k larger, as such products have them."""
    hq, hkv, d = HEADS[case["heads"]]
    g = _gen(seed, tag)
    x = torch.randn(rows, (hq + 2 * hkv) * d, generator=g, device="cuda", dtype=torch.float32)
    big = torch.exp(0.5 * torch.randn(hkv * d, generator=g, device="cuda", dtype=torch.float32))
    x[:, hq * d:(hq + hkv) * d] *= big
    return x.to(kind).unflatten(1, (hq + 2 * hkv, d))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _sums(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _seq_pos(lo, n):
    """(sequence, position) of the positions lo .. lo + n of every sequence, packed."""
    n, lo = torch.as_tensor(n, device="cuda"), torch.as_tensor(lo, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    return seq, torch.arange(len(seq), device="cuda") - (torch.cumsum(n, 0) - n)[seq] + lo[seq]


def _slots(table, page, lo, n):
    seq, pos = _seq_pos(lo, n)
    return table[seq, pos // page].long() * page + pos % page


def _table(counts, n_pages, seed):
    """A page table: counts[i] pages for row i, in random places; the rest of a row is -1."""
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = torch.arange(max(max(counts), 1))
    n = torch.tensor(counts)
    start = torch.cumsum(n, 0) - n
    there = at[None] < n[:, None]
    return torch.where(there, order[torch.where(there, start[:, None] + at[None], 0)], -1).cuda()


def _plan(case):
    """(pairs of each axis, angles' base): an eighth of a head stays as it is where there are several axes."""
    d = HEADS[case["heads"]][2]
    if case["axes"] == 1:
        return [d // 2], 10000.0
    pairs = d // 2 - d // 16
    first = pairs // case["axes"] // 2 if case["axes"] == 3 else pairs // 3
    rest = (pairs - first) // (case["axes"] - 1)
    return [first] + [rest] * (case["axes"] - 2) + [pairs - first - rest * (case["axes"] - 2)], 1000000.0


def _positions(case):
    """Of each new token: its number, and behind every 200 tokens of text an image of 24 x 16 patches, which stand at one time."""
    past, new = _lens(case)
    seq, pos = _seq_pos(past, new)
    if case["axes"] == 1:
        return pos[:, None].to(torch.int32).contiguous()
    place = pos % 584
    image, patch = place >= 200, place - 200
    start = pos // 584 * 224 + torch.clamp(place, max=200)
    axes = [start, start + torch.where(image, patch // 24, 0), start + torch.where(image, patch % 24, 0)]
    return torch.stack(axes[:case["axes"]], 1).to(torch.int32).contiguous()


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


def _logits(case, seed):
    """Logits as an LM head gives them: most of the mass on few tokens, each beam's a little different; running scores."""
    g = _gen(seed, 1)
    s, b, v = case["seqs"], case["beams"], case["vocab"]
    x = torch.randn(s, 1, v, generator=g, device="cuda") * 2.5 + torch.randn(s, b, v, generator=g, device="cuda") * 0.5
    scores = -20 * torch.rand(s, b, generator=g, device="cuda") - 5
    return x.flatten(0, 1).to(TYPES[case["type"]]), scores


def _cache_rows(case, seed, rows):
    """k and v of cached tokens; some channels of k larger."""
    hq, hkv, d = HEADS[case["heads"]]
    g = _gen(seed, 3)
    big = torch.exp(0.5 * torch.randn(hkv * d, generator=g, device="cuda", dtype=torch.float32)).view(hkv, d)
    k = torch.randn(rows, hkv, d, generator=g, device="cuda", dtype=torch.float32) * big
    return k.half(), torch.randn(rows, hkv, d, generator=g, device="cuda", dtype=torch.float32).half()


def _plain_cache(fmt, n, hkv, d):
    if fmt == "f16":
        return {s: torch.zeros(n, hkv, d, dtype=torch.float16, device="cuda") for s in ("k", "v")}
    groups = 1 if fmt == "int8" else d // 32
    kind = torch.float32 if fmt == "int8" else torch.float16
    c = {s: torch.zeros(n, hkv, d, dtype=torch.int8, device="cuda") for s in ("k", "v")}
    return c | {s + "_scale": torch.zeros(n, hkv, groups, dtype=kind, device="cuda") for s in ("k", "v")}


def _page_bytes(case, n_pages, seed):
    """Pages as bytes: [page, head, block of 16 tokens, bytes]."""
    hq, hkv, d = HEADS[case["heads"]]
    return torch.randint(0, 256, (n_pages, hkv, case["page"] // 16, 16 * _token_bytes(case["fmt"], d)), generator=_gen(seed, 2),
                         device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "beam":
        st["logits"], st["scores"] = _logits(case, seed)
        if own:
            from bit_weight_only_gb300 import qgemv
            st["ws"] = qgemv.BeamWorkspace(case["seqs"], case["beams"], case["vocab"], case["width"])
        return st
    hq, hkv, d = HEADS[case["heads"]]
    past, new = _lens(case)
    page = case["page"]
    if case["op"] == "rope":
        sections, base = _plan(case)
        every = [p % page + n for p, n in zip(past, new)]  # the pages that the new tokens are in
        st["rows"] = _stack(case, seed, sum(new), TYPES[case["type"]], 1)
        st["positions"] = _positions(case)
        table = _table([-(-n // page) for n in every], sum(-(-n // page) for n in every) + 2, seed)
        lo = [p % page for p in past]
        st |= {"table": table, "slots": _slots(table, page, lo, new), "starts": _ints(lo), "cu": _ints(_sums(new)), "n": sum(new)}
        if own:
            from bit_weight_only_gb300 import qgemv
            st["rotary"] = qgemv.Rotary(d, sections, base=base, pairs=case["pairs"])
            if case["into"] != "rows":
                st["cache"] = qgemv.KVCache(case["into"], int(table.max()) + 2, page, hkv, d)
        else:
            j = torch.arange(sum(sections), dtype=torch.float64, device="cuda")
            st["freqs"] = torch.exp(-j / sum(sections) * math.log(base))
            st["axis"] = torch.repeat_interleave(torch.arange(len(sections), device="cuda"), torch.tensor(sections, device="cuda"))
            if case["into"] != "rows":
                st["cache"] = _plain_cache(case["into"], (int(table.max()) + 2) * page, hkv, d)
        return st
    if case["op"] in ("fork", "compact"):
        if case["op"] == "fork":
            # a sequence's beams share the pages of its prompt, half of its length, and have their own behind it
            n, lens = case["beams"], [p for p in past for _ in range(case["beams"])]
            mine = [-(-p // page) for p in past]
            n_pages = sum(m // 2 + n * (m - m // 2) for m in mine) + case["seqs"] * n + 3
            table = _table([m for m in mine for _ in range(n)], n * sum(mine) + 1, seed)
            lead = table[torch.arange(len(lens), device="cuda") // n * n]
            shared = torch.arange(table.shape[1], device="cuda") < torch.tensor([m // 2 for m in mine for _ in range(n)], device="cuda")[:, None]
            table = torch.where(shared, lead, table)
            there = table >= 0
            ids, at = torch.unique(table[there], return_inverse=True)  # numbers below n_pages, in random places
            places = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed + 1))[:len(ids)].cuda()
            table = table.clone()
            table[there] = places[at].to(torch.int32)
            st |= {"parents": _ints(_parents(case)), "lens": _ints(lens)}
        else:
            n_pages = case["pages"]
            table = _table([-(-p // page) for p in past], n_pages, seed)
        there = table >= 0
        counts = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        counts.index_add_(0, table[there].long(), torch.ones_like(table[there]))
        st |= {"table": table, "counts": counts, "pages": _page_bytes(case, n_pages, seed)}
        if own:
            from bit_weight_only_gb300 import qgemv
            st["pool"] = qgemv.PagePool(n_pages, page)
            st["cache"] = qgemv.KVCache(case["fmt"], n_pages, page, hkv, d)
            st["cache"].pages.copy_(st.pop("pages").flatten())
        else:
            st["refs"] = torch.zeros_like(counts)
        return st
    # a cache with everything in it, and the summaries of its whole pages
    every = [p + n for p, n in zip(past, new)]
    n_pages = sum(-(-n // page) for n in every) + 3
    table = _table([-(-n // page) for n in every], n_pages, seed)
    whole = [p // page for p in past]
    k, v = _cache_rows(case, seed, sum(every))
    slots = _slots(table, page, [0] * len(past), every)
    seq, at = _seq_pos([0] * len(past), whole)
    full = table[seq, at].contiguous()
    if case["fresh"] == "all":
        fresh = full
    else:
        w = torch.tensor(whole, device="cuda")
        fresh = table[torch.arange(len(past), device="cuda"), (w - 1).clamp(min=0)][w > 0].contiguous()
    st |= {"table": table, "ctx": _ints(past), "cu": _ints(_sums(new)), "max_ctx": max(past), "max_new": max(new), "fresh": fresh,
           "q": _stack(case, seed, sum(new), torch.float16, 5)[:, :hq],
           "masks": torch.tensor([m - (1 << 64 if m >> 63 else 0) for m in _masks(case)], dtype=torch.int64, device="cuda")}
    if own:
        from bit_weight_only_gb300 import qgemv
        st["cache"] = qgemv.KVCache(case["fmt"], n_pages, page, hkv, d)
        st["cache"].write(k, v, slots)
        st["summary"] = qgemv.KeySummary(st["cache"])
        st["summary"].update(full)
        st["ws"] = qgemv.AttnWorkspace(len(new), hq, d)
    else:
        st["cache"] = _plain_cache(case["fmt"], n_pages * page, hkv, d)
        _plain_write(case["fmt"], st["cache"], k, v, slots)
        st["codes"] = torch.zeros(n_pages, hkv, 2, d, dtype=torch.int8, device="cuda")
        st["scales"] = torch.zeros(n_pages, hkv, dtype=torch.float32, device="cuda")
        _plain_summary(st, full)
        n = torch.tensor(new, device="cuda")
        at = torch.arange(max(new), device="cuda")
        there = at[None] < n[:, None]
        st["pad"] = {"rows": torch.where(there, (torch.cumsum(n, 0) - n)[:, None] + at[None], 0), "there": there}
    return st


# ------------------------------------------------------------- plain form --

def _plain_codes(fmt, x):
    x = x.float()
    if fmt == "int8":
        a = x.abs().amax(-1, keepdim=True)
        a = a / torch.full_like(a, 127)  # a division (by a plain number torch multiplies by its reciprocal)
        q = torch.where(a > 0, torch.clamp(torch.round(x / a), -127, 127), torch.zeros_like(x))
        return q.to(torch.int8), a
    b = x.unflatten(-1, (-1, 32))
    a = torch.gather(b, -1, b.abs().argmax(-1, keepdim=True)) / -8
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


def _plain_rotated(st, x):
    """x fp32 [n, heads, d] rotated; the angles in 64 bits."""
    angle = st["positions"].double()[:, st["axis"]] * st["freqs"]
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    n = len(st["freqs"])
    if st["case"]["pairs"] == "halves":
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * c - b * s, a * s + b * c, x[..., 2 * n:]], -1)
    a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), x[..., 2 * n:]], -1)


def _plain_rope(st):
    case = st["case"]
    hq, hkv, d = HEADS[case["heads"]]
    x = st["rows"].float()
    turned = _plain_rotated(st, x[:, :hq + hkv])
    if case["into"] == "rows":
        return {"rows": turned.half()}
    _plain_write(case["into"], st["cache"], turned[:, hq:], x[:, hq + hkv:], st["slots"])
    k, v = (_plain_values(case["into"], st["cache"], s, st["slots"]).half() for s in ("k", "v"))
    return {"q": turned[:, :hq].half(), "k": k, "v": v}


def _plain_beam(st):
    case = st["case"]
    x = st["logits"].double().unflatten(0, (case["seqs"], case["beams"]))
    top = x.amax(-1, keepdim=True)
    lse = top + (x - top).exp().sum(-1, keepdim=True).log()
    score = st["scores"].double()[..., None] - lse
    fine = torch.isfinite(score)
    x = torch.where(fine, x + score, torch.full_like(x, -math.inf)).flatten(1)
    best, at = torch.sort(x, dim=1, descending=True, stable=True)
    best, at = best[:, :case["width"]], at[:, :case["width"]]
    none = best == -math.inf
    return {"scores": best.float(), "beams": torch.where(none, -1, at // case["vocab"]).to(torch.int32),
            "tokens": torch.where(none, -1, at % case["vocab"]).to(torch.int32)}


def _plain_fork(st):
    table, parents, page = st["table"].long(), st["parents"].long(), st["case"]["page"]
    refs, lens = st["refs"], st["lens"].long()
    refs.copy_(st["counts"])
    n, rows, at = len(refs), len(parents), torch.arange(table.shape[1], device="cuda")
    used = -(-lens // page)
    kids = torch.zeros_like(lens).index_add_(0, parents, torch.ones_like(parents))
    part = (at == (used - 1)[:, None]) & (lens % page != 0)[:, None]
    change = torch.where(part, kids.clamp(max=1)[:, None], kids[:, None].expand_as(table)) - 1
    there = (at < used[:, None]) & (table >= 0) & (table < n)
    more = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    more.index_add_(0, torch.where(there, table, n).flatten(), torch.where(there, change, 0).flatten())
    refs += more[:n].to(torch.int32)
    first = torch.full_like(lens, rows).scatter_reduce_(0, parents, torch.arange(rows, device="cuda"), "amin")
    new = torch.where(at < used[:, None], table, -1)[parents]
    last = (used - 1).clamp(min=0)
    src = table[torch.arange(len(lens), device="cuda"), last][parents]
    need = (lens % page != 0)[parents] & (src >= 0) & (first[parents] != torch.arange(rows, device="cuda"))
    free = torch.nonzero(refs <= 0).flatten()
    free = torch.cat([free, torch.full((rows,), -1, device="cuda")])
    dst = torch.where(need, free[torch.where(need, torch.cumsum(need, 0) - 1, 0)], -1)
    refs[dst[dst >= 0]] = 1
    new[torch.nonzero(need).flatten(), last[parents][need]] = dst[need]
    # the tokens of the copied pages, in blocks of 16
    held = -(-(lens % page)[parents] // 16)
    go = need & (dst >= 0)
    block = torch.arange(page // 16, device="cuda") < held[go][:, None]
    pages = st["pages"]
    pages[dst[go]] = torch.where(block[:, None, :, None], pages[src[go]], pages[dst[go]])
    return {"table": new.to(torch.int32), "refs": refs, "pages": pages}


def _plain_compact(st):
    table, refs, pages = st["table"].long(), st["refs"], st["pages"]
    refs.copy_(st["counts"])
    used = refs > 0
    low = torch.arange(len(refs), device="cuda") < used.sum()
    src, dst = torch.nonzero(used & ~low).flatten(), torch.nonzero(~used & low).flatten()
    to = torch.arange(len(refs), device="cuda")
    to[src] = dst
    new = torch.where((table >= 0) & (table < len(refs)), to[table.clamp(0, len(refs) - 1)], table)
    refs[dst] = refs[src]
    refs[src] = 0
    pages[dst] = pages[src]
    return {"table": new.to(torch.int32), "refs": refs, "pages": pages}


def _coded(x):
    """INT8 codes of x [..., n] with the scale max|x| / 127, and the scale."""
    a = x.abs().amax(-1)
    a = a / torch.full_like(a, 127)
    return torch.where(a[..., None] > 0, torch.clamp(torch.round(x / a[..., None]), -127, 127), torch.zeros_like(x)), a


def _plain_summary(st, pages):
    page = st["case"]["page"]
    slots = pages.long()[:, None] * page + torch.arange(page, device="cuda")
    x = _plain_values(st["case"]["fmt"], st["cache"], "k", slots)           # pages, tokens, heads, d
    both = torch.cat([x.amax(1), x.amin(1)], -1)
    codes, a = _coded(both)
    st["codes"][pages.long()] = codes.to(torch.int8).unflatten(-1, (2, -1))
    st["scales"][pages.long()] = a


def _plain_sparse(st):
    case = st["case"]
    hq, hkv, d = HEADS[case["heads"]]
    page, g = case["page"], hq // hkv
    _plain_summary(st, st["fresh"])
    ctx, table = st["ctx"].long(), st["table"].long()
    rows, there = st["pad"]["rows"], st["pad"]["there"]
    seqs, new = rows.shape
    q = torch.where(there[..., None, None], st["q"][rows], 0).unflatten(2, (hkv, g))           # b, t, head, g, d
    parts = torch.cat([q.double().clamp(min=0).sum((1, 3)), q.double().clamp(max=0).sum((1, 3))], -1)
    w = _coded(parts.float())[0]                                                             # b, head, 2 d
    at = torch.arange(table.shape[1], device="cuda")
    whole = ctx // page
    cand = (at < whole[:, None]) & (table >= 0)
    codes = st["codes"][table.clamp(min=0)].flatten(3).float()                                 # b, pages, head, 2 d
    # sums of whole numbers below 2^24: exact in any order
    s = (codes * w[:, None]).sum(-1) * st["scales"][table.clamp(min=0)]
    s = torch.where(cand[..., None], s, torch.full_like(s, -math.inf)).transpose(1, 2)         # b, head, pages
    order = torch.sort(s, dim=-1, descending=True, stable=True)[1][..., :case["select"]]
    count = cand.sum(1).clamp(max=case["select"])
    k = order.shape[-1]
    order = torch.where(torch.arange(k, device="cuda") < count[:, None, None], order, table.shape[1])
    order = torch.sort(order, dim=-1)[0]
    # its own table for each head: the selected pages, then those from the last whole page on
    tail = (2 * page + DRAFTS - 2) // page
    width = case["select"] + tail
    col = torch.arange(width, device="cuda")
    from_tail = whole[:, None] + col - count[:, None]                                          # b, width
    wide = torch.cat([table, torch.full((seqs, width + 1), -1, device="cuda")], 1)
    held = torch.gather(wide, 1, torch.where((col >= count[:, None]) & (col < (count + tail)[:, None]) & (from_tail < table.shape[1]),
                                             from_tail, table.shape[1]))
    picked = torch.gather(wide[:, None].expand(seqs, hkv, -1), 2, order)
    picked = torch.cat([picked, torch.full((seqs, hkv, width - k), -1, device="cuda")], 2)
    own_table = torch.where((col < count[:, None])[:, None], picked, held[:, None].expand(seqs, hkv, width))
    own_ctx = count * page + ctx % page
    # attention over them
    slots = (own_table.clamp(min=0)[..., None] * page + torch.arange(page, device="cuda")).flatten(2)  # b, head, keys
    head = torch.arange(hkv, device="cuda")[None, :, None]
    key, val = (_plain_values(case["fmt"], {n: c.flatten(0, 1) for n, c in st["cache"].items()}, n, slots * hkv + head) for n in ("k", "v"))
    j = torch.arange(width * page, device="cuda") - own_ctx[:, None]                           # b, keys
    n_new = st["cu"].diff().long()
    bit = (st["masks"][rows][:, :, None] >> j.clamp(0, 63)[:, None]) & 1
    see = (j < 0)[:, None] | ((j >= 0) & (j < n_new[:, None]))[:, None] & (bit == 1)             # b, t, keys
    see = see[:, None] & (own_table >= 0).repeat_interleave(page, 2)[:, :, None]               # b, head, t, keys
    s = torch.einsum("bthgd,bhkd->bhtgk", q.float(), key) / math.sqrt(d)
    s = torch.where(see[:, :, :, None], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (s - top).exp()
    n = p.sum(-1, keepdim=True)
    out = torch.einsum("bhtgk,bhkd->bthgd", p / torch.where(n > 0, n, torch.ones_like(n)), val).flatten(2, 3)
    lse = (top + n.log())[..., 0].permute(0, 2, 1, 3).flatten(2)
    return {"out": out[there].half(), "lse": lse[there], "pages": own_table.to(torch.int32)}


# -------------------------------------------------------------------- run --

def run(st):
    case = st["case"]
    if not own:
        return {"rope": _plain_rope, "beam": _plain_beam, "fork": _plain_fork, "compact": _plain_compact, "sparse": _plain_sparse}[case["op"]](st)
    from bit_weight_only_gb300 import qgemv
    if case["op"] == "beam":
        scores, beams, tokens = qgemv.beam_select(st["logits"], st["scores"], case["width"], workspace=st["ws"])
        return {"scores": scores, "beams": beams, "tokens": tokens}
    if case["op"] == "rope":
        hq, hkv, d = HEADS[case["heads"]]
        x = st["rows"]
        if case["into"] == "rows":
            return {"rows": st["rotary"].rotate(x[:, :hq + hkv], st["positions"], dtype=torch.float16)}
        q = st["cache"].write_rotated(st["rotary"], x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], st["positions"], st["slots"])
        k, v = st["cache"].read(st["table"], st["starts"], st["cu"], st["n"])
        return {"q": q, "k": k, "v": v}
    if case["op"] in ("fork", "compact"):
        pool, cache = st["pool"], st["cache"]
        pool.refs.copy_(st["counts"])
        if case["op"] == "fork":
            table, src, dst, tokens = pool.fork(st["table"], st["parents"], st["lens"])
            cache.copy_pages(src, dst, tokens)
        else:
            table, src, dst = pool.compact(st["table"])
            cache.copy_pages(src, dst)
        hkv, d = cache.kv_heads, cache.head_dim
        return {"table": table, "refs": pool.refs, "pages": cache.pages.view(-1, hkv, case["page"] // 16, 16 * _token_bytes(case["fmt"], d))}
    st["summary"].update(st["fresh"])
    pages, lens = st["cache"].select(st["q"], st["table"], st["ctx"], st["cu"], summary=st["summary"], n_select=case["select"])
    out, lse = st["cache"].attend_pages(st["q"], pages, lens, st["cu"], st["masks"], max_ctx=min(st["max_ctx"], (case["select"] + 1) * case["page"]),
                                        max_new=st["max_new"], workspace=st["ws"])
    return {"out": out, "lse": lse, "pages": pages}


# ------------------------------------------------------------------ exact --

def _exact_values(fmt, x):
    """What the cache stands for, in 64 bits; the codes of 32-bit values are decided in 32 bits, by definition."""
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


def _exact_turned(case, x):
    sections, base = _plan(case)
    pos, n = _positions(case).double(), sum(sections)
    axes = sum(([i] * s for i, s in enumerate(sections)), [])
    y = x.double().clone()
    for j in range(n):
        i, k = (j, j + n) if case["pairs"] == "halves" else (2 * j, 2 * j + 1)
        z = torch.polar(torch.ones(len(pos), dtype=torch.float64, device="cuda"), pos[:, axes[j]] * base ** (-j / n))[:, None]
        z = torch.complex(x[..., i].double(), x[..., k].double()) * z
        y[..., i], y[..., k] = z.real, z.imag
    return y


def _exact_sparse(case, seed):
    hq, hkv, d = HEADS[case["heads"]]
    past, new = _lens(case)
    page, g = case["page"], hq // hkv
    k, v = (_exact_values(case["fmt"], x) for x in _cache_rows(case, seed, sum(past) + sum(new)))
    q = _stack(case, seed, sum(new), torch.float16, 5)[:, :hq].double()
    masks = _masks(case)
    out = torch.zeros(sum(new), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(new), hq, dtype=torch.float64, device="cuda")
    a = b = 0
    for p, n in zip(past, new):
        whole = p // page
        for h in range(hkv):
            qq = q[b:b + n, h * g:(h + 1) * g]
            kk, vv = k[a:a + p + n, h], v[a:a + p + n, h]
            keep = torch.ones(p, dtype=torch.bool, device="cuda")
            if whole > case["select"]:
                blocks = kk[:whole * page].float().reshape(whole, page, d)
                edge = torch.cat([blocks.max(1).values, blocks.min(1).values], 1)
                scale = edge.abs().max(1).values / torch.tensor([127.0], device="cuda")
                edge = (edge / scale[:, None]).round().clamp(-127, 127)
                pull = torch.cat([qq.clamp(min=0).sum((0, 1)), qq.clamp(max=0).sum((0, 1))]).float()
                pull = (pull / (pull.abs().max() / torch.tensor([127.0], device="cuda"))).round().clamp(-127, 127)
                score = (edge.double() @ pull.double()).float() * scale
                best = torch.argsort(score, descending=True, stable=True)[:case["select"]]
                keep[:whole * page] = False
                keep[:whole * page].view(whole, page)[best] = True
            see = torch.zeros(n, p + n, dtype=torch.bool, device="cuda")
            see[:, :p] = keep
            see[:, p:] = torch.tensor([[bool(m >> j & 1) for j in range(n)] for m in masks[b:b + n]], device="cuda")
            s = torch.einsum("tgd,kd->tgk", qq, kk) / math.sqrt(d)
            s = s.masked_fill(~see[:, None], -math.inf)
            lse[b:b + n, h * g:(h + 1) * g] = torch.logsumexp(s, -1)
            out[b:b + n, h * g:(h + 1) * g] = torch.softmax(s, -1) @ vv
        a, b = a + p + n, b + n
    return {"out": out, "lse": lse, "pages": None}


def exact(case, seed):
    if case["op"] == "beam":
        x, scores = _logits(case, seed)
        best = []
        for s in range(case["seqs"]):  # a sequence at a time
            rows = torch.log_softmax(x[s * case["beams"]:(s + 1) * case["beams"]].double(), -1) + scores[s].double()[:, None]
            best.append(torch.topk(rows.flatten(), case["width"]).values)
        return {"scores": torch.stack(best), "beams": None, "tokens": None}
    if case["op"] == "rope":
        hq, hkv, d = HEADS[case["heads"]]
        x = _stack(case, seed, sum(_lens(case)[1]), TYPES[case["type"]], 1)
        turned = _exact_turned(case, x[:, :hq + hkv])
        if case["into"] == "rows":
            return {"rows": turned}
        return {"q": turned[:, :hq], "k": _exact_values(case["into"], turned[:, hq:]), "v": _exact_values(case["into"], x[:, hq + hkv:])}
    if case["op"] == "sparse":
        return _exact_sparse(case, seed)
    return None  # pages and their numbers: nothing is computed that has digits
