"""The paged serving operators as measured cases: page tables and slot maps
built from request lengths, the append of new keys and values to the page
cache, and attention over the cache for a batch that may share a prefix.

Each operator is here in a plain form of elementary torch operations
(`own = False`) and as the library's call (`own = True`); `exact` computes the
same from the definition in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a running batch: most requests take no new page
        {"name": "tables_decode_step", "op": "tables", "batch": 64, "page": 16, "width": 512, "new": 1,
         "old_max": 8191, "len_seed": 1},
        # a large batch admitted at once: every table and slot map built from nothing
        {"name": "tables_admit", "op": "tables", "batch": 2048, "page": 16, "width": 1024, "new": 1024,
         "old_max": 0, "len_seed": 2},
        # one new token for each request of a decoding batch
        {"name": "append_decode", "op": "append", "batch": 64, "new": 1, "kv_heads": 8, "dim": 128, "page": 16,
         "ragged": False, "len_seed": 3},
        # the keys and values of ragged prompts, 16 heads
        {"name": "append_prompts", "op": "append", "batch": 16, "new": 2048, "kv_heads": 16, "dim": 128,
         "page": 64, "ragged": True, "len_seed": 4},
        # a single short request: latency
        {"name": "decode_one_short", "op": "attn", "batch": 1, "heads": 8, "kv_heads": 8, "dim": 128, "new": 1,
         "page": 16, "prefix": 0, "own_min": 777, "own_max": 777, "causal": True, "short_q": False, "len_seed": 5},
        # a decoding batch of very unequal lengths, four query heads to a key head
        {"name": "decode_ragged", "op": "attn", "batch": 64, "heads": 32, "kv_heads": 8, "dim": 128, "new": 1,
         "page": 16, "prefix": 0, "own_min": 1, "own_max": 8192, "causal": True, "short_q": False, "len_seed": 6},
        # one request with a very long context
        {"name": "decode_long", "op": "attn", "batch": 1, "heads": 24, "kv_heads": 8, "dim": 128, "new": 1,
         "page": 128, "prefix": 0, "own_min": 131072, "own_max": 131072, "causal": True, "short_q": False,
         "len_seed": 7},
        # a decoding batch whose requests share a long system prompt
        {"name": "decode_prefix", "op": "attn", "batch": 128, "heads": 32, "kv_heads": 8, "dim": 128, "new": 1,
         "page": 64, "prefix": 16333, "own_min": 1, "own_max": 1000, "causal": True, "short_q": False,
         "len_seed": 8},
        # several drafted tokens for each request, checked in one pass
        {"name": "drafts_prefix_d64", "op": "attn", "batch": 32, "heads": 16, "kv_heads": 4, "dim": 64, "new": 5,
         "page": 32, "prefix": 4099, "own_min": 5, "own_max": 1000, "causal": True, "short_q": True,
         "len_seed": 9},
        # pieces of prompts behind a shared prefix
        {"name": "prompt_prefix", "op": "attn", "batch": 4, "heads": 24, "kv_heads": 8, "dim": 128, "new": 1024,
         "page": 128, "prefix": 8192, "own_min": 600, "own_max": 2048, "causal": True, "short_q": True,
         "len_seed": 10},
        # whole prompts without a prefix, as many key heads as query heads
        {"name": "prompt_d64", "op": "attn", "batch": 2, "heads": 16, "kv_heads": 16, "dim": 64, "new": 2048,
         "page": 16, "prefix": 0, "own_min": 2048, "own_max": 2048, "causal": True, "short_q": False,
         "len_seed": 11},
        # an encoder's states kept in pages, read by every query row
        {"name": "states_no_mask", "op": "attn", "batch": 16, "heads": 16, "kv_heads": 16, "dim": 128, "new": 77,
         "page": 16, "prefix": 0, "own_min": 1, "own_max": 1000, "causal": False, "short_q": True,
         "len_seed": 12},
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_one(rng):
    op = rng.choice(("tables", "append", "attn", "attn", "attn"))
    seed = rng.randrange(1 << 20)
    page = rng.choice((16, 32, 64, 128))
    if op == "tables":
        width = _log_int(rng, 4, 2048)
        old = rng.choice((0, rng.randrange(width * page)))
        new = min(_log_int(rng, 1, 2048), width * page - old)
        return {"op": op, "batch": _log_int(rng, 1, 4096), "page": page, "width": width, "new": max(new, 1),
                "old_max": old, "len_seed": seed}
    if op == "append":
        return {"op": op, "batch": _log_int(rng, 1, 256), "new": _log_int(rng, 1, 4096),
                "kv_heads": rng.choice((1, 2, 3, 4, 8, 16, 24)), "dim": rng.choice((64, 128)), "page": page,
                "ragged": rng.random() < 0.5, "len_seed": seed}
    kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
    new = rng.choice((1, 1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 2048)))
    longest = max(new, _log_int(rng, 1, 65536))
    return {"op": op, "batch": _log_int(rng, 1, 256), "heads": kv_heads * rng.choice((1, 1, 2, 3, 4, 8)),
            "kv_heads": kv_heads, "dim": rng.choice((64, 128)), "new": new, "page": page,
            "prefix": rng.choice((0, _log_int(rng, 1, 32768))), "own_min": rng.choice((1, longest)),
            "own_max": longest, "causal": rng.random() < 0.75, "short_q": rng.random() < 0.5, "len_seed": seed}


def _plain_elements(case):
    """Values the plain form of the attention holds at once: scores, and keys and values read from the pages."""
    keys = case["prefix"] + case["own_max"]
    return (case["batch"] * case["heads"] * case["new"] * keys,
            case["kv_heads"] * case["dim"] * (case["batch"] * case["own_max"] + case["prefix"]))


def draw(rng):
    """One more case of the ranges the listed ones stand for, no larger than the largest of its operator."""
    while True:
        case = _draw_one(rng)
        same = [c for c in listed() if c["op"] == case["op"]]
        most = {k: max(work(c)[k] for c in same) for k in ("bytes", "flops")}
        got = work(case)
        if any(got[k] > most[k] for k in most):
            continue
        if case["op"] == "attn":
            scores, values = _plain_elements(case)
            if scores > 1.2e9 or values > 6e8:
                continue
        return case


# ---------------------------------------------------------------------------
# Lengths: part of the case, the same for every seed
# ---------------------------------------------------------------------------
def _lengths(case):
    """What each request holds: (before, after) for the tables, new rows for
    the append, (new rows, own keys) for the attention."""
    r = random.Random(case["len_seed"])
    B = case["batch"]
    if case["op"] == "tables":
        old = [r.randint(0, case["old_max"]) for _ in range(B)]
        if case["new"] == 1:
            return old, [o + 1 for o in old]
        return old, [o + r.randint(1, case["new"]) for o in old]
    if case["op"] == "append":
        return [r.randint(1, case["new"]) if case["ragged"] else case["new"] for _ in range(B)]
    q = [r.randint(1, case["new"]) if case["short_q"] else case["new"] for _ in range(B)]
    kv = [r.randint(case["own_min"], case["own_max"]) for _ in range(B)]
    if case["causal"]:
        kv = [max(n, m) for n, m in zip(q, kv)]       # the new tokens' own keys are in the cache
    return q, kv


def _seen(case):
    """Pairs of a query row and a key it sees, over the batch, for one head."""
    q, kv = _lengths(case)
    pairs = 0
    for n, m in zip(q, kv):
        pairs += n * case["prefix"] + (n * m - n * (n - 1) // 2 if case["causal"] else n * m)
    return pairs


def work(case):
    """Inputs read once and outputs written once."""
    B = case["batch"]
    if case["op"] == "tables":
        old, new = _lengths(case)
        p = case["page"]
        taken = sum(-(-b // p) - -(-a // p) for a, b in zip(old, new))
        kept = sum(-(-a // p) for a in old)
        # lengths, pages taken from the free list, table entries that are not kept, slots
        return {"bytes": 8 * B + 4 * taken + 4 * (B * case["width"] - kept) + 4 * B * case["new"] + 4,
                "flops": B * (case["width"] + case["new"])}
    if case["op"] == "append":
        rows = sum(_lengths(case))
        return {"bytes": 2 * 2 * rows * case["kv_heads"] * case["dim"] * 2 + 4 * B * case["new"], "flops": 0}
    q, kv = _lengths(case)
    H, G, D, p = case["heads"], case["kv_heads"], case["dim"], case["page"]
    rows = 2 * 2 * sum(q) * H * D                                     # Q read, O written
    keys = 2 * 2 * (sum(kv) + case["prefix"]) * G * D
    index = 4 * (sum(-(-n // p) for n in kv) + -(-case["prefix"] // p) + 2 * B + 1)
    return {"bytes": rows + keys + index, "flops": 4 * D * H * _seen(case)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _pool(pages, page, heads, dim, g):
    """A page cache in use: every page holds values of earlier tokens; keys carry an offset for each channel."""
    shape = (pages, page, heads, dim)
    k = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
    k += torch.randn((heads, dim), generator=g, device=DEVICE, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
    # as [page, head, token, channel], which is how the library's views are ordered
    return k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)


def _tables(lengths, page, width, pages, unused=-1):
    """A table row for each length, from the list `pages`."""
    t = torch.full((len(lengths), max(width, 1)), unused, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lengths):
        m = -(-n // page)
        t[b, :m] = pages[at:at + m]
        at += m
    return t


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    c = torch.Generator().manual_seed(seed)
    B, page = case["batch"], case["page"]
    state = {"case": case}
    if case["op"] == "tables":
        old, new = _lengths(case)
        held = sum(-(-n // page) for n in old)
        need = sum(-(-b // page) - -(-a // page) for a, b in zip(old, new))
        order = torch.randperm(held + need + 64, generator=c).to(torch.int32)
        # what earlier requests left in the table's unused entries is still there
        state.update(old_len=_int32(old), new_len=_int32(new), free=order[held:].to(DEVICE),
                     table=_tables(old, page, case["width"], order, unused=held).to(DEVICE),
                     slots=torch.empty((B, case["new"]), dtype=torch.int32, device=DEVICE),
                     taken=torch.empty((1,), dtype=torch.int32, device=DEVICE))
        return state
    if case["op"] == "append":
        n, heads, dim = _lengths(case), case["kv_heads"], case["dim"]
        width = -(-case["new"] // page)
        order = torch.randperm(sum(-(-m // page) for m in n) + 8, generator=c).to(torch.int32)
        table = _tables(n, page, width, order).long()
        at = torch.arange(case["new"])
        slots = table[:, at // page] * page + at % page
        slots = torch.where(at[None] < torch.tensor(n)[:, None], slots, -1)
        # new keys and values as views into one projection's output
        kv = torch.randn((B, case["new"], 2, heads, dim), generator=g, device=DEVICE, dtype=torch.bfloat16)
        state.update(k=kv[:, :, 0].permute(0, 2, 1, 3), v=kv[:, :, 1].permute(0, 2, 1, 3),
                     slots=slots.to(torch.int32).to(DEVICE))
        state["cache_k"], state["cache_v"] = _pool(order.numel(), page, heads, dim, g)
    else:
        q, kv = _lengths(case)
        H, heads, dim, new, pre = case["heads"], case["kv_heads"], case["dim"], case["new"], case["prefix"]
        shared = -(-pre // page)
        order = torch.randperm(shared + sum(-(-m // page) for m in kv) + 8, generator=c).to(torch.int32)
        state.update(
            q=torch.randn((B, new, H, dim), generator=g, device=DEVICE, dtype=torch.bfloat16).permute(0, 2, 1, 3),
            o=torch.zeros((B, new, H, dim), device=DEVICE, dtype=torch.bfloat16).permute(0, 2, 1, 3),
            table=_tables(kv, page, -(-case["own_max"] // page), order[shared:]).to(DEVICE),
            q_len=_int32(q), kv_len=_int32(kv), prefix_table=order[:shared].to(DEVICE) if pre else None,
            prefix_len=_int32([pre]) if pre else None)
        state["cache_k"], state["cache_v"] = _pool(order.numel(), page, heads, dim, g)
    if own:
        import quantized_exact_attention_gb300 as S
        state["cache"] = S.PageCache(state["cache_k"], state["cache_v"])
        if case["op"] == "attn":
            state["workspace"] = S.alloc_paged_workspace(B, case["heads"], case["kv_heads"], case["new"],
                                                         case["dim"], device=DEVICE)
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if case["op"] == "tables":
        return (_own_tables if own else _plain_tables)(state)
    if case["op"] == "append":
        return (_own_append if own else _plain_append)(state)
    return (_own_attn if own else _plain_attn)(state)


def _own_tables(s):
    import quantized_exact_attention_gb300 as S
    S.sage_page_tables(s["new_len"], s["case"]["page"], s["free"], s["table"], s["slots"], s["taken"],
                       old_len=s["old_len"])
    return {"table": s["table"], "slots": s["slots"], "taken": s["taken"]}


def _own_append(s):
    import quantized_exact_attention_gb300 as S
    S.sage_cache_append(s["k"], s["v"], s["slots"], s["cache"])
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _own_attn(s):
    import quantized_exact_attention_gb300 as S
    S.sage_attn_paged(s["q"], s["o"], s["cache"], s["table"], s["workspace"], q_len=s["q_len"],
                      kv_len=s["kv_len"], prefix_table=s["prefix_table"], prefix_len=s["prefix_len"],
                      causal=s["case"]["causal"])
    return s["o"]


def _plain_tables(s):
    page, table = s["case"]["page"], s["table"]
    old_len, new_len = s["old_len"], s["new_len"]
    old_pages, new_pages = (old_len + page - 1) // page, (new_len + page - 1) // page
    need = new_pages - old_pages
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=DEVICE)
    take = col - old_pages[:, None] + first[:, None]
    fresh = (col >= old_pages[:, None]) & (col < new_pages[:, None]) & (take < s["free"].numel())
    picked = s["free"][take.clamp(0, s["free"].numel() - 1)]
    table = torch.where(col < old_pages[:, None], table, torch.where(fresh, picked, -1))
    pos = old_len[:, None] + torch.arange(s["case"]["new"], device=DEVICE)
    at = torch.gather(table, 1, (pos // page).clamp(max=table.shape[1] - 1).long())
    slots = torch.where((pos < new_len[:, None]) & (at >= 0), at * page + pos % page, -1)
    return {"table": table.to(torch.int32), "slots": slots.to(torch.int32),
            "taken": need.sum().to(torch.int32).reshape(1)}


def _plain_append(s):
    page = s["case"]["page"]
    live = (s["slots"] >= 0).nonzero(as_tuple=True)
    slot = s["slots"][live].long()
    for new, cache in ((s["k"], s["cache_k"]), (s["v"], s["cache_v"])):
        cache.permute(0, 2, 1, 3)[slot // page, slot % page] = new.permute(0, 2, 1, 3)[live]
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _read_pages(cache, table):
    """Keys or values of table [..., pages] in 32 bits: [..., head, token, channel]."""
    x = cache[table.clamp(min=0).long()].float()                     # [..., pages, head, token, channel]
    x = x.transpose(-4, -3)
    return x.reshape(x.shape[:-3] + (x.shape[-3] * x.shape[-2], x.shape[-1]))


def _plain_attn(s):
    case = s["case"]
    B, H, heads, N, D = case["batch"], case["heads"], case["kv_heads"], case["new"], case["dim"]
    G = H // heads
    q = s["q"].float().reshape(B, heads, G * N, D)
    k, v = _read_pages(s["cache_k"], s["table"]), _read_pages(s["cache_v"], s["table"])
    key = torch.arange(k.shape[2], device=DEVICE)
    row = torch.arange(N, device=DEVICE)
    last = s["kv_len"][:, None] - 1                                   # last key row i sees
    if case["causal"]:
        last = row[None] + (s["kv_len"] - s["q_len"])[:, None]
    sees = (key[None, None] <= last[:, :, None]) & (key[None, None] < s["kv_len"][:, None, None])
    scores = torch.matmul(q, k.transpose(-1, -2)).reshape(B, heads, G, N, -1) * (1.0 / math.sqrt(D))
    scores.masked_fill_(~sees[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    if s["prefix_table"] is not None:
        pk, pv = _read_pages(s["cache_k"], s["prefix_table"]), _read_pages(s["cache_v"], s["prefix_table"])
        rows = q.transpose(0, 1).reshape(heads, B * G * N, D)         # every request's rows meet the prefix at once
        pre = torch.matmul(rows, pk.transpose(-1, -2)).reshape(heads, B, G, N, -1) * (1.0 / math.sqrt(D))
        pre.masked_fill_(torch.arange(pk.shape[1], device=DEVICE) >= s["prefix_len"], -math.inf)
        top = torch.maximum(top, pre.amax(-1, keepdim=True).transpose(0, 1))
    top = torch.where(top == -math.inf, 0.0, top)
    weight = torch.exp_(scores.sub_(top))
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.reshape(B, heads, G * N, -1), v).reshape(B, heads, G, N, D)
    del scores, weight
    if s["prefix_table"] is not None:
        weight = torch.exp_(pre.sub_(top.transpose(0, 1)))
        total = total + weight.sum(-1, keepdim=True).transpose(0, 1)
        out = out + torch.matmul(weight.reshape(heads, B * G * N, -1), pv).reshape(heads, B, G, N, D).transpose(0, 1)
    out = torch.where(total > 0, out / total, 0.0).reshape(B, H, N, D)
    out = torch.where((row[None] < s["q_len"][:, None])[:, None, :, None], out, 0.0)
    return out.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# The same from the definition, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        page, table, free = case["page"], s["table"].cpu().tolist(), s["free"].cpu().tolist()
        slots, taken = [], 0
        for b, (a, n) in enumerate(zip(*_lengths(case))):
            row = table[b]
            for j in range(-(-a // page), case["width"]):
                row[j] = -1
            for j in range(-(-a // page), -(-n // page)):
                row[j] = free[taken]
                taken += 1
            slots.append([row[t // page] * page + t % page if t < n else -1 for t in range(a, a + case["new"])])
        return {"table": _int32(table), "slots": _int32(slots), "taken": _int32([taken])}
    if case["op"] == "append":
        page, B, n = case["page"], case["batch"], _lengths(case)
        out = {}
        for name in ("k", "v"):
            cache = s["cache_" + name].double().permute(0, 2, 1, 3).contiguous()
            flat = cache.reshape(-1, case["kv_heads"], case["dim"])
            for b in range(B):
                flat[s["slots"][b, :n[b]].long()] = s[name][b, :, :n[b]].double().transpose(0, 1)
            out[name] = flat.reshape(cache.shape).permute(0, 2, 1, 3)
        return out
    q_len, kv_len = _lengths(case)
    page, G, D, pre = case["page"], case["heads"] // case["kv_heads"], case["dim"], case["prefix"]
    out = torch.zeros((case["batch"], case["heads"], case["new"], D), dtype=torch.float64, device=DEVICE)

    def tokens(cache, h, pages, n):
        return cache[pages.long(), h].reshape(-1, D)[:n].double()

    for h in range(case["kv_heads"]):
        shared = [tokens(s["cache_" + x], h, s["prefix_table"], pre) for x in "kv"] if pre else None
        for b, (n, m) in enumerate(zip(q_len, kv_len)):
            k, v = (tokens(s["cache_" + x], h, s["table"][b, :-(-m // page)], m) for x in "kv")
            hidden = torch.zeros((n, m), dtype=torch.bool, device=DEVICE)
            if case["causal"]:
                hidden = torch.arange(m, device=DEVICE)[None] > torch.arange(n, device=DEVICE)[:, None] + (m - n)
            if pre:
                k, v = torch.cat((shared[0], k)), torch.cat((shared[1], v))
                hidden = torch.cat((torch.zeros((n, pre), dtype=torch.bool, device=DEVICE), hidden), 1)
            x = torch.einsum("gnd,md->gnm", s["q"][b, h * G:(h + 1) * G, :n].double(), k) / math.sqrt(D)
            x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[b, h * G:(h + 1) * G, :n] = x @ v
    return out
