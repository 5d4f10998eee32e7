"""The operators of a tree of drafted tokens served from the page cache, as
measured cases: visibility words and depths from the tree's parents, rotary
positions of queries and gradients, the append that rotates keys on their way
into the cache, attention of the tree's tokens over the cache, and the move of
the accepted tokens to the front.

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
        # the drafted trees of a small running batch, before a step's first layer
        {"name": "tree_tables_step", "op": "tables", "batch": 8, "tokens": 26, "width": 4, "ragged": True,
         "len_seed": 1},
        # a large batch of wide trees; the last words of a row are partly used
        {"name": "tree_tables_batch", "op": "tables", "batch": 1024, "tokens": 250, "width": 12, "ragged": False,
         "len_seed": 2},
        # queries of one new token for each request of a decoding batch, from the requests' lengths
        {"name": "rope_decode", "op": "rope", "batch": 64, "heads": 32, "tokens": 1, "dim": 128, "rotary": 128,
         "interleaved": False, "base": 500000.0, "stretch": 1.0, "far": 8191, "packed": 0, "inverse": False,
         "ragged": False, "len_seed": 3},
        # the gradient of a long sequence's queries, several documents packed into it, half of each head rotated,
        # frequencies stretched for far positions
        {"name": "rope_gradient", "op": "rope", "batch": 1, "heads": 24, "tokens": 16384, "dim": 128, "rotary": 64,
         "interleaved": True, "base": 10000.0, "stretch": 32.0, "far": 1 << 20, "packed": 5000, "inverse": True,
         "ragged": False, "len_seed": 4},
        # one new token for each request of a decoding batch
        {"name": "append_rope_decode", "op": "append", "batch": 64, "kv_heads": 8, "tokens": 1, "dim": 128, "page": 16,
         "rotary": 128, "interleaved": False, "base": 500000.0, "stretch": 1.0, "far": 8191, "packed": 0,
         "ragged": False, "len_seed": 5},
        # the keys and values of ragged prompts, 16 heads
        {"name": "append_rope_prompts", "op": "append", "batch": 16, "kv_heads": 16, "tokens": 2048, "dim": 128,
         "page": 64, "rotary": 128, "interleaved": False, "base": 10000.0, "stretch": 8.0, "far": 100000, "packed": 0,
         "ragged": True, "len_seed": 6},
        # one request, a small tree: latency
        {"name": "tree_attn_one", "op": "attn", "batch": 1, "heads": 8, "kv_heads": 8, "dim": 128, "tokens": 8,
         "width": 2, "page": 16, "prefix": 0, "own_min": 777, "own_max": 777, "ragged": False, "len_seed": 7},
        # a batch of unequal lengths, four query heads to a key head
        {"name": "tree_attn_batch", "op": "attn", "batch": 32, "heads": 32, "kv_heads": 8, "dim": 128, "tokens": 26,
         "width": 4, "page": 64, "prefix": 0, "own_min": 26, "own_max": 8192, "ragged": True, "len_seed": 8},
        # small trees behind a shared system prompt
        {"name": "tree_attn_prefix_d64", "op": "attn", "batch": 24, "heads": 16, "kv_heads": 4, "dim": 64,
         "tokens": 13, "width": 3, "page": 32, "prefix": 4099, "own_min": 13, "own_max": 1000, "ragged": True,
         "len_seed": 9},
        # very wide trees of few requests with long contexts
        {"name": "tree_attn_wide", "op": "attn", "batch": 4, "heads": 24, "kv_heads": 8, "dim": 128, "tokens": 251,
         "width": 25, "page": 128, "prefix": 0, "own_min": 9000, "own_max": 16384, "ragged": False, "len_seed": 10},
        # what a step of a decoding batch accepted
        {"name": "keep_step", "op": "keep", "batch": 64, "kv_heads": 8, "dim": 128, "tokens": 26, "kept": 6,
         "page": 16, "len_seed": 11},
        # long accepted paths of a large batch
        {"name": "keep_batch", "op": "keep", "batch": 512, "kv_heads": 16, "dim": 128, "tokens": 61, "kept": 20,
         "page": 64, "len_seed": 12},
    ]


def _log_int(rng, lo, hi):
    """A whole number spread over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rotary(rng):
    dim = rng.choice((64, 128))
    return {"dim": dim, "rotary": rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= dim] + [dim] * 3),
            "interleaved": rng.random() < 0.5, "base": rng.choice((10000.0, 500000.0, 1000000.0)),
            "stretch": rng.choice((1.0, 1.0, 4.0, 32.0)), "far": _log_int(rng, 1, 1 << 20)}


def _draw_one(rng):
    op = rng.choice(("tables", "rope", "append", "attn", "attn", "keep"))
    seed = rng.randrange(1 << 20)
    if op == "tables":
        n = _log_int(rng, 1, 512)
        return {"op": op, "batch": _log_int(rng, 1, 1024), "tokens": n, "width": _log_int(rng, 1, max(1, n // 2)),
                "ragged": rng.random() < 0.5, "len_seed": seed}
    if op == "rope":
        n = _log_int(rng, 1, 16384)
        return {"op": op, "batch": _log_int(rng, 1, 256), "heads": _log_int(rng, 1, 64), "tokens": n,
                **_draw_rotary(rng), "packed": rng.choice((0, _log_int(rng, 1, n))),
                "inverse": rng.random() < 0.5, "ragged": rng.random() < 0.5, "len_seed": seed}
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        n = _log_int(rng, 1, 4096)
        return {"op": op, "batch": _log_int(rng, 1, 256), "kv_heads": rng.choice((1, 2, 3, 4, 8, 16, 24)), "tokens": n,
                "page": page, **_draw_rotary(rng), "packed": rng.choice((0, _log_int(rng, 1, n))),
                "ragged": rng.random() < 0.5, "len_seed": seed}
    kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
    if op == "keep":
        n = _log_int(rng, 2, 256)
        return {"op": op, "batch": _log_int(rng, 1, 512), "kv_heads": kv_heads, "dim": rng.choice((64, 128)),
                "tokens": n, "kept": _log_int(rng, 1, n // 2), "page": page, "len_seed": seed}
    n = rng.choice((_log_int(rng, 1, 16), _log_int(rng, 8, 64), _log_int(rng, 17, 256)))
    longest = max(n, _log_int(rng, 1, 65536))
    return {"op": op, "batch": _log_int(rng, 1, 128), "heads": kv_heads * rng.choice((1, 1, 2, 3, 4, 8)),
            "kv_heads": kv_heads, "dim": rng.choice((64, 128)), "tokens": n, "width": _log_int(rng, 1, max(1, n // 2)),
            "page": page, "prefix": rng.choice((0, _log_int(rng, 1, 32768))), "own_min": rng.choice((1, longest)),
            "own_max": longest, "ragged": rng.random() < 0.5, "len_seed": seed}


def _plain_elements(case):
    """Values the plain form of the attention holds at once: scores, and keys and values read from the pages."""
    keys = case["prefix"] + case["own_max"]
    return (case["batch"] * case["heads"] * case["tokens"] * keys,
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
    """What each request holds: new tokens; for the attention (new tokens, own keys); for the move (accepted
    tokens, drafted tokens)."""
    r = random.Random(case["len_seed"])
    B, N = case["batch"], case["tokens"]
    if case["op"] == "keep":
        return [r.randint(1, case["kept"]) for _ in range(B)], [N] * B
    n = [r.randint(1, N) if case["ragged"] else N for _ in range(B)]
    if case["op"] != "attn":
        return n
    return n, [max(m, r.randint(case["own_min"], case["own_max"])) for m in n]


def _level(i, width):
    """Depth of token i of a tree that holds one root and then `width` tokens on each level."""
    return 0 if i == 0 else 1 + (i - 1) // width


def work(case):
    """Inputs read once and outputs written once."""
    B, N = case["batch"], case["tokens"]
    if case["op"] == "tables":
        words = -(-N // 32)
        return {"bytes": 4 * sum(_lengths(case)) + 4 * B + 4 * B * N * (words + 1), "flops": B * N * words}
    if case["op"] == "rope":
        rows = sum(_lengths(case))
        H, D, R = case["heads"], case["dim"], case["rotary"]
        return {"bytes": 2 * 2 * rows * H * D + 4 * B + (4 * rows if case["packed"] else 0) + 4 * R,
                "flops": 3 * rows * H * R}
    if case["op"] == "append":
        rows = sum(_lengths(case))
        H, D, R = case["kv_heads"], case["dim"], case["rotary"]
        return {"bytes": 2 * 2 * 2 * rows * H * D + 4 * B * N + 4 * B + (4 * rows if case["packed"] else 0) + 4 * R,
                "flops": 3 * rows * H * R}
    if case["op"] == "keep":
        kept, _ = _lengths(case)
        moved = sum(k - 1 for k in kept)                   # the root is in place
        return {"bytes": 2 * 2 * 2 * moved * case["kv_heads"] * case["dim"] + 4 * (B * case["kept"] + 2 * moved),
                "flops": 0}
    q, kv = _lengths(case)
    H, G, D, p = case["heads"], case["kv_heads"], case["dim"], case["page"]
    seen = sum(n * (case["prefix"] + m - n) + sum(_level(i, case["width"]) + 1 for i in range(n))
               for n, m in zip(q, kv))
    rows = 2 * 2 * sum(q) * H * D                                     # Q read, O written
    keys = 2 * 2 * (sum(kv) + case["prefix"]) * G * D
    index = 4 * (sum(-(-n // p) for n in kv) + -(-case["prefix"] // p) + 2 * B + 1) + 4 * sum(n * -(-n // 32) for n in q)
    return {"bytes": rows + keys + index, "flops": 4 * D * H * seen}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _frequencies(case):
    """(radians a position for each pair, factor of the rotated channels) in 64 bits: base^(-2 j / R), and for far
    positions those that turn less than once within 8,192 positions divided by `stretch`, those that turn more than
    32 times kept, the others in between."""
    R, s = case["rotary"], case["stretch"]
    plain = [case["base"] ** (-2.0 * j / R) for j in range(R // 2)]
    if s == 1.0:
        return plain, 1.0
    keep = [min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1.0) / 31.0)) for f in plain]
    return [f * k + f / s * (1.0 - k) for f, k in zip(plain, keep)], 0.1 * math.log(s) + 1.0


def _parents(case, g):
    """Parents [B, N] of the drafted tokens: each has one of the level before as its parent."""
    N, width = case["tokens"], case["width"]
    first = torch.tensor([1 + (_level(i, width) - 2) * width if i > width else 0 for i in range(N)], device=DEVICE)
    many = torch.tensor([width if i > width else 1 for i in range(N)], device=DEVICE)
    pick = torch.randint(1 << 30, (case["batch"], N), generator=g, device=DEVICE) % many
    parents = first + pick
    parents[:, 0] = -1
    return parents.to(torch.int32)


def _sees(parents):
    """Truth values [B, N, N]: token i sees token t, itself or one of its ancestors."""
    B, N = parents.shape
    sees = torch.eye(N, dtype=torch.bool, device=DEVICE).expand(B, N, N).clone()
    up, steps = parents.long(), 1
    while steps < N:                                       # ancestors up to `steps` away, then twice as many
        at = up.clamp(min=0)
        sees |= torch.gather(sees, 1, at[:, :, None].expand(B, N, N)) & (up >= 0)[:, :, None]
        up = torch.where(up >= 0, torch.gather(up, 1, at), -1)
        steps *= 2
    return sees


def _words(sees):
    """Truth values [..., N] as int32 words, 32 to a word, the lowest bit first."""
    N = sees.shape[-1]
    padded = torch.nn.functional.pad(sees, (0, -N % 32)).reshape(sees.shape[:-1] + (-1, 32)).long()
    w = (padded << torch.arange(32, device=DEVICE)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _positions(case, g):
    """(start of each request, offsets [B, N] within it or None): the offsets restart where another document begins."""
    start = torch.randint(case["far"] + 1, (case["batch"],), generator=g, device=DEVICE).to(torch.int32)
    if not case["packed"]:
        return start, None
    shift = torch.randint(case["packed"], (case["batch"], 1), generator=g, device=DEVICE)
    return start, ((torch.arange(case["tokens"], device=DEVICE) + shift) % case["packed"]).to(torch.int32)


def _pool(pages, page, heads, dim, g):
    """A page cache in use: every page holds values of earlier tokens; keys carry an offset for each channel."""
    shape = (pages, page, heads, dim)
    k = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
    k += torch.randn((heads, dim), generator=g, device=DEVICE, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
    # as [page, head, token, channel], which is how the library's views are ordered
    return k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)


def _tables(lengths, page, width, pages):
    """A table row for each length, from the list `pages`."""
    t = torch.full((len(lengths), max(width, 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lengths):
        m = -(-n // page)
        t[b, :m] = pages[at:at + m]
        at += m
    return t


def _slots(lengths, tokens, page, order):
    """The slots [B, N] of each request's tokens, -1 behind its length."""
    table = _tables(lengths, page, -(-tokens // page), order).long()
    at = torch.arange(tokens)
    slots = table[:, at // page] * page + at % page
    return torch.where(at[None] < torch.tensor(lengths)[:, None], slots, -1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    c = torch.Generator().manual_seed(seed)
    B, N = case["batch"], case["tokens"]
    state = {"case": case}
    if case["op"] == "tables":
        state.update(parents=_parents(case, g), n_len=_int32(_lengths(case)),
                     mask=torch.empty((B, N, -(-N // 32)), dtype=torch.int32, device=DEVICE),
                     depth=torch.empty((B, N), dtype=torch.int32, device=DEVICE))
    elif case["op"] == "rope":
        shape = (B, N, case["heads"], case["dim"])
        state["x"] = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16).permute(0, 2, 1, 3)
        state["out"] = torch.zeros(shape, device=DEVICE, dtype=torch.bfloat16).permute(0, 2, 1, 3)
        state["n_len"] = _int32(_lengths(case)) if case["ragged"] else None
        state["start"], state["positions"] = _positions(case, g)
    elif case["op"] == "append":
        n, heads, dim, page = _lengths(case), case["kv_heads"], case["dim"], case["page"]
        order = torch.randperm(sum(-(-m // page) for m in n) + 8, generator=c).to(torch.int32)
        # new keys and values as views into one projection's output
        kv = torch.randn((B, N, 2, heads, dim), generator=g, device=DEVICE, dtype=torch.bfloat16)
        state.update(k=kv[:, :, 0].permute(0, 2, 1, 3), v=kv[:, :, 1].permute(0, 2, 1, 3),
                     slots=_slots(n, N, page, order).to(DEVICE))
        state["cache_k"], state["cache_v"] = _pool(order.numel(), page, heads, dim, g)
        state["start"], state["positions"] = _positions(case, g)
    elif case["op"] == "keep":
        kept, n = _lengths(case)
        page = case["page"]
        order = torch.randperm(sum(-(-m // page) for m in n) + 8, generator=c).to(torch.int32)
        # the root, then tokens in rising order from behind the places they go to
        paths = torch.full((B, case["kept"]), -1, dtype=torch.int32)
        r = random.Random(seed)
        for b, k in enumerate(kept):
            paths[b, 0] = 0
            paths[b, 1:k] = torch.tensor(sorted(r.sample(range(case["kept"], N), k - 1)), dtype=torch.int32)
        state.update(slots=_slots(n, N, page, order).to(DEVICE), kept=paths.to(DEVICE))
        state["cache_k"], state["cache_v"] = _pool(order.numel(), page, case["kv_heads"], case["dim"], g)
    else:
        q, kv = _lengths(case)
        H, heads, dim, pre, page = case["heads"], case["kv_heads"], case["dim"], case["prefix"], case["page"]
        shared = -(-pre // page)
        order = torch.randperm(shared + sum(-(-m // page) for m in kv) + 8, generator=c).to(torch.int32)
        state.update(
            q=torch.randn((B, N, H, dim), generator=g, device=DEVICE, dtype=torch.bfloat16).permute(0, 2, 1, 3),
            o=torch.zeros((B, N, H, dim), device=DEVICE, dtype=torch.bfloat16).permute(0, 2, 1, 3),
            table=_tables(kv, page, -(-max(case["own_max"], N) // page), order[shared:]).to(DEVICE),
            mask=_words(_sees(_parents(case, g))), q_len=_int32(q), kv_len=_int32(kv),
            prefix_table=order[:shared].to(DEVICE) if pre else None, prefix_len=_int32([pre]) if pre else None)
        state["cache_k"], state["cache_v"] = _pool(order.numel(), page, heads, dim, g)
    if case["op"] in ("rope", "append"):
        state["frequencies"], state["amplitude"] = _frequencies(case)
        state["f64"] = torch.tensor(state["frequencies"], dtype=torch.float64, device=DEVICE)
    if own:
        import quantized_exact_attention_gb300 as S
        if case["op"] in ("rope", "append"):
            state["rotary_plan"] = S.make_rotary(state["frequencies"], interleaved=case["interleaved"],
                                                 amplitude=state["amplitude"], device=DEVICE)
        if "cache_k" in state:
            state["cache"] = S.PageCache(state["cache_k"], state["cache_v"])
        if case["op"] == "attn":
            state["workspace"] = S.alloc_paged_workspace(B, case["heads"], case["kv_heads"], N, case["dim"],
                                                         device=DEVICE)
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "append": _own_append, "attn": _own_attn,
                "keep": _own_keep}[op](state)
    return {"tables": _plain_tables, "rope": _plain_rope, "append": _plain_append, "attn": _plain_attn,
            "keep": _plain_keep}[op](state)


def _own_tables(s):
    import quantized_exact_attention_gb300 as S
    S.sage_tree_tables(s["parents"], s["mask"], s["depth"], n_len=s["n_len"])
    return {"mask": s["mask"], "depth": s["depth"]}


def _own_rope(s):
    import quantized_exact_attention_gb300 as S
    S.sage_rope(s["x"], s["out"], s["rotary_plan"], positions=s["positions"], start=s["start"], n_len=s["n_len"],
                inverse=s["case"]["inverse"])
    return s["out"]


def _own_append(s):
    import quantized_exact_attention_gb300 as S
    S.sage_cache_append_rope(s["k"], s["v"], s["slots"], s["cache"], s["rotary_plan"], positions=s["positions"],
                             start=s["start"])
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _own_attn(s):
    import quantized_exact_attention_gb300 as S
    S.sage_attn_paged_tree(s["q"], s["o"], s["cache"], s["table"], s["mask"], s["workspace"], q_len=s["q_len"],
                           kv_len=s["kv_len"], prefix_table=s["prefix_table"], prefix_len=s["prefix_len"])
    return s["o"]


def _own_keep(s):
    import quantized_exact_attention_gb300 as S
    S.sage_cache_keep(s["kept"], s["slots"], s["cache"])
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _plain_tables(s):
    N = s["case"]["tokens"]
    live = torch.arange(N, device=DEVICE)[None] < s["n_len"][:, None]
    sees = _sees(s["parents"]) & live[:, :, None]
    depth = torch.where(live, sees.sum(-1) - 1, 0)
    return {"mask": _words(sees), "depth": depth.to(torch.int32)}


def _plain_turned(x, s):
    """x [B, H, N, D] in 32 bits with its first channels rotated."""
    case = s["case"]
    R, half = case["rotary"], case["rotary"] // 2
    at = s["positions"] if s["positions"] is not None else torch.arange(case["tokens"], device=DEVICE)[None]
    at = (s["start"][:, None] + at).double()
    angle = at[:, None, :, None] * s["f64"]                            # [B, 1, N, R / 2]
    cos, sin = ((f(angle) * s["amplitude"]).float() for f in (torch.cos, torch.sin))
    if case.get("inverse"):
        sin = -sin
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).reshape(y.shape[:-1] + (R,))
    else:
        a, b = y[..., :half], y[..., half:R]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, y[..., R:]), -1)


def _plain_rope(s):
    y = _plain_turned(s["x"], s).to(torch.bfloat16)
    if s["n_len"] is None:
        return y
    live = torch.arange(y.shape[2], device=DEVICE)[None] < s["n_len"][:, None]
    return torch.where(live[:, None, :, None], y, s["out"])


def _plain_append(s):
    page = s["case"]["page"]
    live = (s["slots"] >= 0).nonzero(as_tuple=True)
    slot = s["slots"][live].long()
    for new, cache in ((_plain_turned(s["k"], s).to(torch.bfloat16), s["cache_k"]), (s["v"], s["cache_v"])):
        cache.permute(0, 2, 1, 3)[slot // page, slot % page] = new.permute(0, 2, 1, 3)[live]
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _plain_keep(s):
    page, kept = s["case"]["page"], s["kept"].long()
    to = s["slots"][:, :kept.shape[1]]
    move = kept >= 0
    src, dst = torch.gather(s["slots"], 1, kept.clamp(min=0))[move].long(), to[move].long()
    for cache in (s["cache_k"], s["cache_v"]):
        rows = cache.permute(0, 2, 1, 3)
        rows[dst // page, dst % page] = rows[src // page, src % page]
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _read_pages(cache, table):
    """Keys or values of table [..., pages] in 32 bits: [..., head, token, channel]."""
    x = cache[table.clamp(min=0).long()].float()                     # [..., pages, head, token, channel]
    x = x.transpose(-4, -3)
    return x.reshape(x.shape[:-3] + (x.shape[-3] * x.shape[-2], x.shape[-1]))


def _plain_attn(s):
    case = s["case"]
    B, H, heads, N, D = case["batch"], case["heads"], case["kv_heads"], case["tokens"], case["dim"]
    G = H // heads
    q = s["q"].float().reshape(B, heads, G * N, D)
    k, v = _read_pages(s["cache_k"], s["table"]), _read_pages(s["cache_v"], s["table"])
    key = torch.arange(k.shape[2], device=DEVICE)
    row = torch.arange(N, device=DEVICE)
    new = key[None] - (s["kv_len"] - s["q_len"])[:, None]             # [B, keys]: which new token a key is of
    word = torch.gather(s["mask"], 2, (new.clamp(0, N - 1) // 32)[:, None].expand(B, N, -1))
    bit = (word >> (new.clamp(0, N - 1) % 32)[:, None]) & 1
    sees = ((new[:, None] < 0) | (bit > 0)) & (key[None, None] < s["kv_len"][:, None, None])
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
def _exact_sets(parents):
    """For each token of one tree the tokens it sees, as the bits of a whole number."""
    sets = []
    for i, p in enumerate(parents):
        sets.append((1 << i) | (sets[p] if p >= 0 else 0))
    return sets


def _exact_turned(x, s):
    """x [B, H, N, D] in 64 bits: a pair of channels is a complex number, turned by its angle."""
    case = s["case"]
    R = case["rotary"]
    x = x.double()
    first = x[..., :R]
    pairs = first.unflatten(-1, (-1, 2)) if case["interleaved"] else first.unflatten(-1, (2, -1)).transpose(-1, -2)
    steps = torch.arange(case["tokens"], dtype=torch.float64, device=DEVICE).expand(case["batch"], -1)
    if s["positions"] is not None:
        steps = s["positions"].double()
    angle = (s["start"].double()[:, None] + steps)[..., None] * s["f64"]
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), -angle if case.get("inverse") else angle)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    turned = turned.flatten(-2) if case["interleaved"] else turned.transpose(-1, -2).flatten(-2)
    return torch.cat((turned, x[..., R:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        N, words = case["tokens"], -(-case["tokens"] // 32)
        mask, depth = [], []
        for parents, n in zip(s["parents"].cpu().tolist(), _lengths(case)):
            sets = _exact_sets(parents[:n])
            depth.append([x.bit_count() - 1 for x in sets] + [0] * (N - n))
            rows = [[(x >> 32 * w) & 0xFFFFFFFF for w in range(words)] for x in sets] + [[0] * words] * (N - n)
            mask.append(rows)
        wide = torch.tensor(mask, dtype=torch.int64, device=DEVICE)
        return {"mask": torch.where(wide >> 31 == 1, wide - (1 << 32), wide).to(torch.int32), "depth": _int32(depth)}
    if case["op"] == "rope":
        y, n = _exact_turned(s["x"], s), _lengths(case)
        for b, m in enumerate(n):
            y[b, :, m:] = 0.0
        return y
    if case["op"] == "append":
        page, n = case["page"], _lengths(case)
        out = {}
        for name, new in (("k", _exact_turned(s["k"], s)), ("v", s["v"].double())):
            cache = s["cache_" + name].double().permute(0, 2, 1, 3).contiguous()
            flat = cache.reshape(-1, case["kv_heads"], case["dim"])
            for b in range(case["batch"]):
                flat[s["slots"][b, :n[b]].long()] = new[b, :, :n[b]].transpose(0, 1)
            out[name] = flat.reshape(cache.shape).permute(0, 2, 1, 3)
        return out
    if case["op"] == "keep":
        kept, slots, out = s["kept"].cpu().tolist(), s["slots"].cpu().tolist(), {}
        src = [slots[b][t] for b, row in enumerate(kept) for t in row if t >= 0]
        dst = [slots[b][i] for b, row in enumerate(kept) for i, t in enumerate(row) if t >= 0]
        for name in ("k", "v"):
            cache = s["cache_" + name].double().permute(0, 2, 1, 3).contiguous()
            flat = cache.reshape(-1, case["kv_heads"], case["dim"])
            flat[_int32(dst).long()] = flat[_int32(src).long()]
            out[name] = flat.reshape(cache.shape).permute(0, 2, 1, 3)
        return out
    q_len, kv_len = _lengths(case)
    page, G, D, pre = case["page"], case["heads"] // case["kv_heads"], case["dim"], case["prefix"]
    out = torch.zeros((case["batch"], case["heads"], case["tokens"], D), dtype=torch.float64, device=DEVICE)
    words = s["mask"].cpu().tolist()
    hidden = []
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        h = torch.zeros((n, pre + m), dtype=torch.bool, device=DEVICE)
        h[:, pre + m - n:] = torch.tensor([[not (words[b][i][t // 32] >> t % 32) & 1 for t in range(n)]
                                           for i in range(n)], device=DEVICE)
        hidden.append(h)

    def tokens(cache, h, pages, n):
        return cache[pages.long(), h].reshape(-1, D)[:n].double()

    for h in range(case["kv_heads"]):
        shared = [tokens(s["cache_" + x], h, s["prefix_table"], pre) for x in "kv"] if pre else None
        for b, (n, m) in enumerate(zip(q_len, kv_len)):
            k, v = (tokens(s["cache_" + x], h, s["table"][b, :-(-m // page)], m) for x in "kv")
            if pre:
                k, v = torch.cat((shared[0], k)), torch.cat((shared[1], v))
            x = torch.einsum("gnd,md->gnm", s["q"][b, h * G:(h + 1) * G, :n].double(), k) / math.sqrt(D)
            x = torch.softmax(x.masked_fill(hidden[b], -math.inf), -1)
            out[b, h * G:(h + 1) * G, :n] = x @ v
    return out
