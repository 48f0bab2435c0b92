"""The operators between two decoding steps of a beam search or of parallel samples over a paged
key/value cache, as cases that can be timed and compared.

Selecting the next beams from the logits; giving each row the pages of the row it continues
(`fork`), finding pages for the new tokens and own copies of pages that several rows would write
(`reserve`), giving pages back (`release`), moving pages' contents (`copy`), and moving the used
pages to the front of the pool (`compact`). `run` computes them from elementary torch operations,
or, where `own` is true, with the framework's kernels.

A page table [rows, max_pages] holds page numbers, -1 where a row has no page; ref_counts [n_pages]
is how many entries of tables name each page, 0 for a free one. The lowest free pages are taken first.
"""
import math

import torch

own = False

END = 2  # the end token of the selections
CODES = tuple(m * s for s in (1.0, -1.0) for m in (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0))


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one sentence, the paper's beam of 4: the smallest call, all latency
        {"name": "select one sentence", "op": "select", "B": 1, "beams": 4, "V": 32000, "pad": 0, "f32": False, "end": True},
        # a batch of sentences, an odd vocabulary without padding: rows start at any even address
        {"name": "select odd vocabulary", "op": "select", "B": 32, "beams": 4, "V": 32003, "pad": 0, "f32": False, "end": True},
        # logits in 32 bits, padded rows, no end token
        {"name": "select f32", "op": "select", "B": 13, "beams": 5, "V": 50001, "pad": 7, "f32": True, "end": False},
        # a full batch at a large vocabulary: the largest selection
        {"name": "select large vocabulary", "op": "select", "B": 64, "beams": 8, "V": 150000, "pad": 0, "f32": False, "end": True},
        # a step of beam search at Transformer-base's decoder: 6 layers, 8 heads of 64
        {"name": "beam step base", "op": "step", "kind": "beam", "groups": 32, "size": 4, "len_min": 2, "len_max": 256, "page": 16,
         "layers": 6, "h_kv": 8, "d": 64, "q4": False},
        # long hypotheses, eight beams each, two layers' pools in one call
        {"name": "beam step long", "op": "step", "kind": "beam", "groups": 48, "size": 8, "len_min": 400, "len_max": 3500, "page": 32,
         "layers": 2, "h_kv": 4, "d": 128, "q4": False},
        # each prompt continued by 15 samples, over a cache of 4-bit codes
        {"name": "samples 4-bit", "op": "step", "kind": "sample", "groups": 8, "size": 16, "len_min": 900, "len_max": 16001, "page": 64,
         "layers": 4, "h_kv": 8, "d": 128, "q4": True},
        # one token more for each of a serving batch: a few new pages out of a nearly full pool
        {"name": "reserve a step", "op": "reserve", "rows": 256, "new": 1, "len_min": 1, "len_max": 4096, "page": 16, "n_pages": 65536},
        # the prompts of 64 sequences at once
        {"name": "reserve prompts", "op": "reserve", "rows": 64, "new": 8192, "len_min": 1001, "len_max": 8192, "page": 16,
         "n_pages": 262144},
        # whole pages of four layers, as when a prompt's pages are moved: the largest case
        {"name": "copy pages", "op": "copy", "copies": 2500, "page": 16, "layers": 4, "h_kv": 8, "d": 128, "q4": False},
        # a small pool after a batch of sentences
        {"name": "compact small pool", "op": "compact", "rows": 24, "len_min": 1, "len_max": 300, "page": 16, "n_pages": 700,
         "layers": 6, "h_kv": 8, "d": 64, "q4": False},
        # a 4-bit pool of which three quarters are free
        {"name": "compact 4-bit", "op": "compact", "rows": 128, "len_min": 100, "len_max": 4000, "page": 32, "n_pages": 33001,
         "layers": 2, "h_kv": 4, "d": 128, "q4": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.25 / hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "step", "step", "reserve", "copy", "compact"])
    if op == "select":
        beams, f32 = rng.randint(1, 16), rng.random() < 0.3
        V = _log_int(rng, 40, 160000)
        most = 70_000_000 // (2 if f32 else 1)  # logits in all
        return {"op": op, "B": _log_int(rng, 1, max(1, min(200, most // (beams * V)))), "beams": beams, "V": V,
                "pad": rng.choice([0, 0, 1, 7, (-V) % 8]), "f32": f32, "end": rng.random() < 0.8}
    shape = {"page": rng.choice([16, 32, 64, 128]), "h_kv": rng.choice([1, 2, 3, 4, 5, 8]), "d": rng.choice([64, 128]),
             "q4": rng.random() < 0.4, "layers": rng.randint(1, 6)}
    row = shape["layers"] * 2 * shape["h_kv"] * (shape["d"] * (0.6 if shape["q4"] else 2))  # bytes of a row in all layers
    if op == "copy":
        return {"op": op, "copies": _log_int(rng, 1, max(1, min(4000, int(5e8 / (row * shape["page"]))))), **shape}
    if op == "reserve":
        rows, page = _log_int(rng, 1, 600), shape["page"]
        new = _log_int(rng, 1, 8192)
        top = new + _log_int(rng, 1, 4096) - 1
        need = rows * (top // page + 1)
        return {"op": op, "rows": rows, "new": new, "len_min": _log_int(rng, 1, top), "len_max": top, "page": page,
                "n_pages": need + _log_int(rng, 16, 200000)}
    if op == "compact":
        rows = _log_int(rng, 1, 200)
        top = _log_int(rng, 1, max(1, min(4096, int(1e8 / (row * rows)))))
        used = rows * (top // shape["page"] + 1)
        return {"op": op, "rows": rows, "len_min": _log_int(rng, 1, top), "len_max": top,
                "n_pages": used + _log_int(rng, 1, max(1, min(40000, int(5e8 / (row * shape["page"]))))), **shape}
    groups, size = _log_int(rng, 1, 64), rng.randint(1, 16)
    top = _log_int(rng, 1, max(1, min(16384, int(3e8 / (row * groups * (0.4 * size + 0.6))))))
    return {"op": op, "kind": rng.choice(["beam", "sample"]), "groups": groups, "size": size, "len_min": _log_int(rng, 1, top),
            "len_max": top, **shape}


def _spread(n, lo, hi):
    """n whole numbers over lo .. hi, the largest first."""
    return [hi - int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(n)]


def _step_rows(case):
    """Of each row of a step: its length before the new token, how many new tokens (none or one), and the row it continues.
    Beams: the first 1 + g % size beams of sentence g go on, the others are replaced by one of them. Samples: a
    group's first row is the prompt, which gets no token, the others continue it."""
    size, lens, new, parents = case["size"], [], [], []
    for g, length in enumerate(_spread(case["groups"], case["len_min"], case["len_max"])):
        kept = 1 + g % size if case["kind"] == "beam" else 1
        lens += [length] * size
        new += [1] * size if case["kind"] == "beam" else [0] + [1] * (size - 1)
        parents += [g * size + j % kept for j in range(size)]
    return lens, new, parents


def _row_bytes(case):
    d = case["d"]
    return 2 * case["layers"] * case["h_kv"] * (d // 2 + d // 16 if case["q4"] else 2 * d)


def work(case):
    op = case["op"]
    if op == "select":
        live = sum(1 if b % 8 == 7 else case["beams"] for b in range(case["B"]))  # at a sentence's start one beam is alive
        return {"bytes": live * case["V"] * (4 if case["f32"] else 2) + 40 * case["B"] * case["beams"], "flops": 4 * live * case["V"]}
    page = case["page"]
    if op == "copy":
        rows = sum(page if i % 4 else 1 + i % page for i in range(case["copies"]))
        return {"bytes": 2 * rows * _row_bytes(case) + 12 * case["copies"], "flops": 0}
    if op == "reserve":
        lens, new = _reserve_rows(case)
        got = sum(-(-L // page) - -(-(L - m) // page) for L, m in zip(lens, new))
        return {"bytes": 4 * case["n_pages"] + 8 * case["rows"] + 16 * got, "flops": 0}
    if op == "compact":
        used = [-(-L // page) for L in _spread(case["rows"], case["len_min"], case["len_max"])]
        moved = sum(used) * (1 - sum(used) / case["n_pages"])  # of pages at random places
        return {"bytes": 8 * case["n_pages"] + 8 * sum(used) + 2 * moved * page * _row_bytes(case), "flops": 0}
    lens, new, parents = _step_rows(case)
    own_row = [b == p for b, p in enumerate(parents)]
    table = 4 * sum(-(-L // page) * (1 if o else 2) for L, o in zip(lens, own_row))
    rows = sum(L % page for L, o in zip(lens, own_row) if not o)
    return {"bytes": table + 12 * len(lens) + 2 * rows * _row_bytes(case), "flops": 0}


# ------------------------------------------------------------------ inputs

def _reserve_rows(case):
    """Lengths with the new tokens, and how many are new."""
    lens = _spread(case["rows"], case["len_min"], case["len_max"])
    return lens, [min(L, case["new"]) for L in lens]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pool(case, n_pages, gen):
    shape = (case["layers"], n_pages, case["h_kv"], case["page"])
    d = case["d"]
    if not case["q4"]:
        return {n: torch.randn(shape + (d,), generator=gen, device="cuda", dtype=torch.bfloat16) for n in ("k", "v")}
    pool = {}
    for n in ("k", "v"):
        pool[n + "_codes"] = torch.randint(0, 256, shape + (d // 2,), generator=gen, device="cuda", dtype=torch.uint8)
        pool[n + "_scales"] = torch.randint(0, 127, shape + (d // 16,), generator=gen, device="cuda", dtype=torch.uint8)
    return pool


def _table(rows_pages, max_pages, n_pages, gen):
    """A page table whose rows name the given slots (lists of numbers below n_pages), the slots being pages in a random
    order, and the counts."""
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    slots = torch.full((len(rows_pages), max_pages), -1, dtype=torch.int64)
    for b, slot in enumerate(rows_pages):
        slots[b, :len(slot)] = torch.tensor(slot, dtype=torch.int64)
    slots = slots.cuda()
    table = torch.where(slots >= 0, order[slots.clamp(min=0)], -1)
    counts = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
    counts.index_add_(0, torch.where(table >= 0, table, n_pages).flatten(), torch.ones_like(table).flatten())
    return table.contiguous(), counts[:n_pages].clone()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "select":
        B, K, V, stride = case["B"], case["beams"], case["V"], case["V"] + case["pad"]
        # most tokens unlikely, a few of each row likely, the end token sometimes among them
        x = 2 * torch.randn(B * K, stride, generator=gen, device="cuda") - 4
        few = torch.randint(0, V, (B * K, 6), generator=gen, device="cuda")
        x.scatter_add_(1, few, 4 + 3 * torch.randn(B * K, 6, generator=gen, device="cuda").abs())
        if V > END:
            x[:, END] += 12 * (torch.rand(B * K, generator=gen, device="cuda") < 0.4)
        s["x"] = x.to(torch.float32 if case["f32"] else torch.bfloat16)
        first = torch.arange(B, device="cuda")[:, None] % 8 == 7
        dead = first & (torch.arange(K, device="cuda") > 0)
        scores = -60 * torch.rand(B, 1, generator=gen, device="cuda") - 4 * torch.rand(B, K, generator=gen, device="cuda")
        s["scores"] = torch.where(dead, -math.inf, scores).contiguous()
        s["lengths"] = torch.randint(1, 100, (B,), generator=gen, device="cuda", dtype=torch.int32)
        past = -0.2 - 3 * torch.rand(B, K, generator=gen, device="cuda")
        s["ended"] = torch.where(first | (torch.rand(B, K, generator=gen, device="cuda") < 0.5), -math.inf, past).sort(dim=1, descending=True).values.contiguous()
        s["ended_rows"] = torch.randint(0, B * K, (B, K), generator=gen, device="cuda", dtype=torch.int32)
        s["ended_lengths"] = torch.randint(1, 100, (B, K), generator=gen, device="cuda", dtype=torch.int32)
        s["tokens"], s["parents"] = torch.empty(B, K, dtype=torch.int32, device="cuda"), torch.empty(B, K, dtype=torch.int32, device="cuda")
        s["new_scores"] = torch.empty(B, K, device="cuda")
        if own:  # a program keeps its workspace
            import transformer_scaled_dot_gb300 as tsd
            s["bytes"] = tsd.beam_select_workspace_bytes(B, K, V)
            s["workspace"] = torch.empty(s["bytes"], dtype=torch.uint8, device="cuda")
        return s
    page = case["page"]
    if op == "copy":
        n, n_pages = case["copies"], 2 * case["copies"] + 3
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        rows = _ints([page if i % 4 else 1 + i % page for i in range(n)])
        s |= {"n_pages": n_pages, "copies": torch.stack([order[:n], order[n:2 * n], rows], 1).contiguous(), "n_copies": _ints([n]),
              "most": n, "pool": _pool(case, n_pages, gen)}
        return s
    if op == "reserve":
        lens, new = _reserve_rows(case)
        slots, at = [], 0
        for L, m in zip(lens, new):
            slots.append(range(at, at + -(-(L - m) // page)))
            at += len(slots[-1])
        max_pages = -(-case["len_max"] // page) + 1
        s["table"], s["counts"] = _table(slots, max_pages, case["n_pages"], gen)
        # most of the pool belongs to other tables
        short = sum(-(-L // page) for L in lens)
        others = (s["counts"] == 0).float() * torch.rand(case["n_pages"], generator=gen, device="cuda")
        taken = int(0.9 * max(0, case["n_pages"] - short))
        if taken:
            s["counts"][others.topk(taken).indices] = 1
        s |= {"lens": _ints(lens), "new_lens": _ints(new), "keep": _ints([L - m for L, m in zip(lens, new)]), "B": len(lens),
              "n_new": case["new"], "max_pages": max_pages}
    elif op == "compact":
        slots, at = [], 0
        for L in _spread(case["rows"], case["len_min"], case["len_max"]):
            slots.append(range(at, at + -(-L // page)))
            at += len(slots[-1])
        max_pages = max(len(x) for x in slots) + 1
        s["table"], s["counts"] = _table(slots, max_pages, case["n_pages"], gen)
        s |= {"table_out": torch.empty_like(s["table"]), "counts_out": torch.empty_like(s["counts"]), "B": case["rows"],
              "max_pages": max_pages, "most": min(at, case["n_pages"]), "n_used": _ints([0]), "pool": _pool(case, case["n_pages"], gen)}
    else:
        lens, new, parents = _step_rows(case)
        size, slots, at = case["size"], [], 0
        for b, L in enumerate(lens):
            used = -(-L // page)
            if b % size == 0:  # the group's common start
                common = range(at, at + (int(0.6 * (L // page)) if case["kind"] == "beam" else used))
                at += len(common)
            if case["kind"] == "sample":
                slots.append(common if b % size == 0 else [])
            else:
                slots.append([*common, *range(at, at + used - len(common))])
                at += used - len(common)
        max_pages = -(-(case["len_max"] + 1) // page) + 1
        s["n_pages"] = at + 2 * len(lens) + 3
        s["table"], s["counts"] = _table(slots, max_pages, s["n_pages"], gen)
        s |= {"lens": _ints([L + m for L, m in zip(lens, new)]), "new_lens": _ints(new), "parents": _ints(parents), "B": len(lens),
              "n_new": 1, "max_pages": max_pages, "most": len(lens), "pool": _pool(case, s["n_pages"], gen)}
    s["copies"] = torch.full((s.get("most", s["B"]), 3), -1, dtype=torch.int32, device="cuda")
    s["n_copies"], s["n_missing"] = _ints([0]), _ints([0])
    if own:
        import transformer_scaled_dot_gb300 as tsd
        s["bytes"] = tsd.attn_cache_pages_workspace_bytes(s["B"], s["n_pages"])
        s["workspace"] = torch.empty(s["bytes"], dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms

def _best(x, n):
    """The n largest of each row of x, equal ones by their place: values and places."""
    value, at = x.topk(n)
    last = value[:, -1:]
    place = torch.arange(x.shape[1], device="cuda")
    equal = torch.where(x == last, place, x.shape[1]).topk(n, largest=False).values
    at = torch.cat([torch.where(value > last, at, x.shape[1]), equal], 1).sort(dim=1).values  # by place
    value = torch.where(at < x.shape[1], x.gather(1, at.clamp(max=x.shape[1] - 1)), -math.inf)
    value, order = value.sort(dim=1, descending=True, stable=True)
    return value[:, :n], at.gather(1, order)[:, :n]


def _select(s):
    B, K, V, end = s["B"], s["beams"], s["V"], s["end"]
    x = s["x"][:, :V].double()  # totals that lie next to one another decide: 64 bits
    top = x.amax(1, keepdim=True)
    total = (top + (x - top).exp().sum(1, keepdim=True).log()).neg_().add(s["scores"].view(-1, 1)) + x
    value, at = _best(torch.where(s["scores"].view(-1, 1) > -math.inf, total, -math.inf).view(B, K * V), min(2 * K if end else K, K * V))
    row, token = at // V + K * torch.arange(B, device="cuda")[:, None], at % V
    real = value > -math.inf
    ends = real & (token == END) if end else torch.zeros_like(real)
    goes = real & ~ends
    place = torch.where(goes, (goes.cumsum(1) - 1).clamp(max=K), K)
    for out, new, none in ((s["tokens"], token.int(), END if end else 0), (s["new_scores"], value.float(), -math.inf),
                           (s["parents"], row.int(), torch.arange(B * K, dtype=torch.int32, device="cuda").view(B, K))):
        full = torch.empty(B, K + 1, dtype=out.dtype, device="cuda")
        full[:, :K] = none
        out.copy_(full.scatter_(1, place, new)[:, :K])
    if end:
        lengths = s["lengths"][:, None]
        score = torch.where(ends, value / ((5.0 + lengths.double()) / 6.0) ** 0.6, -math.inf).float()
        score, order = torch.cat([s["ended"], score], 1).sort(dim=1, descending=True, stable=True)
        rows = torch.cat([s["ended_rows"], row.int()], 1).gather(1, order)[:, :K]
        at = torch.cat([s["ended_lengths"], lengths.expand_as(ends)], 1).gather(1, order)[:, :K]
        s["ended"].copy_(score[:, :K])
        # a place that no hypothesis takes keeps what it held
        taken = score[:, :K] > -math.inf
        s["ended_rows"].copy_(torch.where(taken, rows, s["ended_rows"]))
        s["ended_lengths"].copy_(torch.where(taken, at, s["ended_lengths"]))
    return _selected(s)


def _selected(s):
    out = {n: s[n] for n in ("tokens", "parents", "new_scores")}
    return out | {n: s[n] for n in ("ended", "ended_rows", "ended_lengths")} if s["end"] else out


def _count(counts, table, where, by):
    """Adds `by` to the count of every page that `table` names where `where` holds."""
    padded = torch.cat([counts, counts.new_zeros(1)])
    padded.index_add_(0, torch.where(where, table, len(counts)).flatten(), torch.full_like(table, by).flatten())
    counts.copy_(padded[:-1])


def _fork(s):
    table, parents = s["table"], s["parents"]
    new = table[parents.long()]
    changed = new != table
    _count(s["counts"], new, changed & (new >= 0), 1)
    _count(s["counts"], table, changed & (table >= 0), -1)
    table.copy_(new)


def _release(s):
    table = s["table"]
    drop = (torch.arange(s["max_pages"], device="cuda") >= -(-s["keep"] // s["page"])[:, None]) & (table >= 0)
    _count(s["counts"], table, drop, -1)
    table.copy_(torch.where(drop, -1, table))


def _reserve(s):
    table, counts, page, n_pages = s["table"], s["counts"], s["page"], len(s["counts"])
    k, b = torch.arange(s["max_pages"], device="cuda"), torch.arange(s["B"], device="cuda", dtype=torch.int32)[:, None]
    before = s["lens"] - s["new_lens"]
    written = (k >= (before // page)[:, None]) & (k < -(-s["lens"] // page)[:, None])
    held = table >= 0
    named = torch.cat([counts, counts.new_zeros(1)])[torch.where(held, table, n_pages).long()]
    shared = written & held & (named > 1)
    # the first of the rows that write a page keeps it, if nobody else names it
    to = torch.where(shared, table, n_pages).flatten().long()
    writers = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda").index_add_(0, to, shared.int().flatten())
    first = torch.full((n_pages + 1,), s["B"], dtype=torch.int32, device="cuda").scatter_reduce_(0, to, b.expand_as(table).flatten(), "amin")
    at = table.clamp(min=0).long()
    leaves = shared & ~((writers[at] == named) & (first[at] == b))
    need = (written & ~held) | leaves
    free = (counts == 0).nonzero().flatten().int()
    rank = need.flatten().cumsum(0).view_as(need) - 1
    total = need.sum()
    enough = total <= len(free)
    need, leaves = need & enough, leaves & enough
    s["n_missing"].copy_((total - len(free)).clamp(min=0).int().view(1))
    fresh = torch.cat([free, free.new_full((1,), -1)])[rank.clamp(0, len(free))]
    copied = leaves & (k == (before // page)[:, None]) & (before % page > 0)[:, None]
    rows = (before % page)[:, None].expand_as(table)
    got = torch.stack([table[copied], fresh[copied], rows[copied]], 1)
    s["copies"][:len(got)] = got
    s["n_copies"].fill_(len(got))
    _count(counts, table, leaves, -1)
    _count(counts, fresh, need, 1)
    table.copy_(torch.where(need, fresh, table))


def _copy(s):
    src, dst, rows = s["copies"][torch.arange(s["most"], device="cuda") < s["n_copies"]].long().unbind(1)
    kept = (torch.arange(s["page"], device="cuda") < rows[:, None])[:, None, :, None]
    for x in s["pool"].values():
        x[:, dst] = torch.where(kept, x[:, src], x[:, dst])


def _compact(s):
    counts, n = s["counts"], len(s["counts"])
    used, page = counts > 0, torch.arange(n, device="cuda")
    total = used.sum()
    src = (used & (page >= total)).nonzero().flatten().flip(0)
    dst = (~used & (page < total)).nonzero().flatten()
    to = page.clone()
    to[src] = dst
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].int(), s["table"]))
    out = counts.clone()
    out[dst], out[src] = counts[src], 0
    s["counts_out"].copy_(out)
    s["copies"][:len(src)] = torch.stack([src, dst, torch.full_like(src, s["page"])], 1).int()
    s["n_copies"].fill_(len(src))
    s["n_used"].copy_(total.int().view(1))


# ------------------------------------------------------------------ one pass

def _done(s):
    """What the page operators leave behind. Codes and scales are moved, never computed: their bytes."""
    op = s["op"]
    names = {"copy": (), "reserve": ("table", "counts", "n_missing"), "compact": ("table_out", "counts_out", "n_used", "copies", "n_copies"),
             "step": ("table", "counts", "copies", "n_copies", "n_missing")}[op]
    return {n: s[n] for n in names} | s.get("pool", {})


def _own(s):
    import transformer_scaled_dot_gb300 as tsd
    op = s["op"]
    if op == "select":
        call = tsd.beam_select_f32 if s["f32"] else tsd.beam_select
        call(s["x"], s["V"] + s["pad"], s["scores"], s["lengths"], s["B"], s["beams"], s["V"], END if s["end"] else -1, 0.6,
             s["tokens"], s["parents"], s["new_scores"], s["ended"], s["ended_rows"], s["ended_lengths"], s["workspace"], s["bytes"])
        return _selected(s)
    if op == "step":
        tsd.attn_cache_fork(s["table"], None, s["counts"], s["parents"], s["B"], s["n_pages"], s["max_pages"])
    if op == "reserve":
        tsd.attn_cache_release(s["table"], s["counts"], s["keep"], s["B"], s["n_pages"], s["page"], s["max_pages"])
    if op in ("step", "reserve"):
        tsd.attn_cache_reserve(s["table"], s["counts"], s["lens"], s["new_lens"], s["copies"], s["n_copies"], s["n_missing"], s["B"],
                               s["n_new"], s["n_pages"], s["page"], s["max_pages"], s["workspace"], s["bytes"])
    if op == "compact":
        tsd.attn_cache_compact(s["table"], s["counts"], s["table_out"], s["counts_out"], s["copies"], s["n_copies"], s["n_used"], s["B"],
                               s["n_pages"], s["page"], s["max_pages"], s["most"], s["workspace"], s["bytes"])
    if op != "reserve":
        p = s["pool"]
        sizes = (s["copies"], s["n_copies"], s["most"], s["layers"], s["n_pages"] * s["h_kv"] * s["page"], s["h_kv"], s["d"], s["n_pages"], s["page"])
        if s["q4"]:
            tsd.attn_cache_copy_q4(p["k_codes"], p["k_scales"], p["v_codes"], p["v_scales"], *sizes)
        else:
            tsd.attn_cache_copy(p["k"], p["v"], *sizes)
    return _done(s)


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "select":
        return _select(s)
    if op == "step":
        _fork(s)
    if op == "reserve":
        _release(s)
    if op in ("step", "reserve"):
        _reserve(s)
    if op == "compact":
        _compact(s)
    if op != "reserve":
        _copy(s)
    return _done(s)


# ------------------------------------------------------------------ the definitions, one thing at a time

def _exact_select(s):
    B, K, V = s["B"], s["beams"], s["V"]
    out = {n: s[n].double() if s[n].is_floating_point() else s[n].long() for n in ("tokens", "parents", "new_scores", "ended", "ended_rows", "ended_lengths")}
    for b in range(B):
        found = []
        for j in range(K):
            score = float(s["scores"][b, j])
            if score == -math.inf:
                continue
            x = s["x"][b * K + j, :V].double()
            p = x - torch.logsumexp(x, 0) + score
            least = p.topk(min(V, 2 * K)).values[-1]
            some = (p >= least).nonzero().flatten()
            found += [(-v, j * V + t) for v, t in zip(p[some].tolist(), some.tolist())]
        found = sorted(found)[:2 * K if s["end"] else K]
        goes = [(-v, at) for v, at in found if not (s["end"] and at % V == END)]
        for j in range(K):
            v, at = goes[j] if j < len(goes) else (-math.inf, j * V + (END if s["end"] else 0))
            out["new_scores"][b, j], out["tokens"][b, j], out["parents"][b, j] = v, at % V, b * K + at // V
        if s["end"]:
            length = int(s["lengths"][b])
            old = [(float(v), int(r), int(n)) for v, r, n in zip(s["ended"][b], s["ended_rows"][b], s["ended_lengths"][b])]
            old += [(-v / ((5 + length) / 6) ** 0.6, b * K + at // V, length) for v, at in found if at % V == END]
            for j, (v, r, n) in enumerate(sorted(old, key=lambda e: -e[0])[:K]):
                out["ended"][b, j] = v
                if v > -math.inf:
                    out["ended_rows"][b, j], out["ended_lengths"][b, j] = r, n
    return out if s["end"] else {n: out[n] for n in ("tokens", "parents", "new_scores")}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op, page = case["op"], case.get("page")
    if op == "select":
        return _exact_select(s)
    copies = []
    if op == "copy":
        copies = s["copies"].tolist()
        out = {}
    elif op == "compact":
        table, counts = s["table"].tolist(), s["counts"].tolist()
        total = sum(c > 0 for c in counts)
        holes = [p for p in range(total) if counts[p] == 0]
        for src in range(len(counts) - 1, total - 1, -1):
            if counts[src]:
                dst = holes[len(copies)]
                copies.append([src, dst, page])
                counts[dst], counts[src] = counts[src], 0
        to = {c[0]: c[1] for c in copies}
        out = {"table_out": torch.tensor([[to.get(p, p) for p in row] for row in table]), "counts_out": torch.tensor(counts), "n_used": _ints([total])}
    else:
        table, counts = s["table"].tolist(), s["counts"].tolist()

        def name(b, k, p):
            if table[b][k] >= 0:
                counts[table[b][k]] -= 1
            table[b][k] = p
            if p >= 0:
                counts[p] += 1

        if op == "step":
            old = [list(row) for row in table]
            for b, parent in enumerate(s["parents"].tolist()):
                for k, p in enumerate(old[parent]):
                    name(b, k, p)
        else:
            for b, keep in enumerate(s["keep"].tolist()):
                for k in range(-(-keep // page), s["max_pages"]):
                    name(b, k, -1)
        lens, new = s["lens"].tolist(), s["new_lens"].tolist()
        wanted = [(b, k) for b in range(s["B"]) for k in range((lens[b] - new[b]) // page, -(-lens[b] // page))]
        writers = {}
        for b, k in wanted:
            if table[b][k] >= 0:
                writers.setdefault(table[b][k], []).append(b)
        moves = []
        for b, k in wanted:
            p = table[b][k]
            if p < 0 or (counts[p] > 1 and not (len(writers[p]) == counts[p] and writers[p][0] == b)):
                moves.append((b, k, p))
        free = [p for p, c in enumerate(counts) if c == 0]
        for (b, k, p), fresh in zip(moves, free):
            rows = (lens[b] - new[b]) - k * page
            if p >= 0 and rows > 0:
                copies.append([p, fresh, rows])
            name(b, k, fresh)
        out = {"table": torch.tensor(table), "counts": torch.tensor(counts), "n_missing": _ints([max(0, len(moves) - len(free))])}
    if op in ("step", "compact"):
        listed_copies = s["copies"].clone()
        if copies:
            listed_copies[:len(copies)] = _ints(copies)
        out |= {"copies": listed_copies, "n_copies": _ints([len(copies)])}
    for src, dst, rows in copies:
        for x in s.get("pool", {}).values():
            x[:, dst, :, :rows] = x[:, src, :, :rows]
    return out | s.get("pool", {})
