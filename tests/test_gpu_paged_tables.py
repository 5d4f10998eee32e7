"""Page tables, slot maps and the append against their definitions (whole
numbers and moved values: equal, not near)."""
import random

import pytest
import torch

import quantized_exact_attention_gb300 as S
from tests import gpu_support as G
from tests import paged_support as P

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call_tables(old, new, page, free, W, N, table=None, pad=0):
    """The library's (table, slots, taken); rows `pad` entries further apart, which stay as they were."""
    G.ensure_built()
    B = len(new)
    wide = torch.full((B, W + pad), 99, dtype=torch.int32, device="cuda")
    t = wide[:, :W]
    if table is not None:
        t.copy_(i32(table))
    swide = torch.full((B, N + pad), 98, dtype=torch.int32, device="cuda")
    s = swide[:, :N]
    taken = S.sage_page_tables(i32(new), page, i32(free), t, s if N else None,
                               old_len=i32(old) if old is not None else None)
    torch.cuda.synchronize()
    assert bool((wide[:, W:] == 99).all()) and bool((swide[:, N:] == 98).all())
    assert S.sage_last_launch_count() == 1
    return t.tolist(), s.tolist(), taken.tolist()


CASES = [
    # B, page, W, N, old_max, new_max, short (free pages missing)
    (1, 16, 1, 1, 0, 1, 0),
    (3, 16, 4, 7, 0, 64, 0),
    (5, 32, 9, 33, 200, 60, 0),
    (2, 128, 3, 300, 0, 384, 0),
    (257, 16, 5, 3, 70, 3, 0),
    (1300, 64, 7, 5, 300, 130, 0),                         # more requests than blocks
    (2000, 16, 4, 2, 62, 2, 13),                           # ... and too few free pages
    (6, 16, 8, 20, 100, 28, 4),
    (4, 16, 300, 4000, 0, 4800, 0),                        # several passes of a block over a row
    (9, 16, 12, 24, 130, 60, 0),
    (1300, 32, 8, 8, 220, 30, 6),
    (3, 128, 2000, 4, 250000, 5, 0),
    (5, 64, 8, 0, 100, 300, 0),                            # no slots
]


# pad: with rows a multiple of 4 long and apart, entries are written in fours
@pytest.mark.parametrize("pad", [3, 4])
@pytest.mark.parametrize("B,page,W,N,old_max,new_max,short", CASES)
def test_tables_from_lengths(B, page, W, N, old_max, new_max, short, pad):
    r = random.Random(B * 1000 + W)
    old = [r.randint(0, old_max) for _ in range(B)]
    new = [o + r.randint(0, new_max) for o in old]
    held = sum(-(-o // page) for o in old)
    need = sum(-(-n // page) - -(-o // page) for o, n in zip(old, new))
    pages = list(range(held + need))
    r.shuffle(pages)
    table = [[-5] * W for _ in range(B)]
    for b, o in enumerate(old):
        for j in range(-(-o // page)):
            table[b][j] = pages.pop()
    free = pages[:max(0, len(pages) - short)]
    got = call_tables(old, new, page, free, W, N, table, pad)
    want = P.tables_reference(old, new, page, free, table, N)
    assert got[0] == want[0]
    assert got[1] == want[1]
    assert got[2] == [want[2]] == [need]
    # the same call on its own output changes nothing
    again = call_tables(old, new, page, free, W, N, got[0], pad)
    assert again == got


def test_lengths_out_of_range_are_clamped_and_none_counts_as_zero():
    page, W, N = 16, 3, 50
    old, new = [-7, 40, 1000, 5], [20, 10, 2000, -3]
    table = [[100 + 10 * b + j for j in range(W)] for b in range(4)]
    free = list(range(20))
    assert call_tables(old, new, page, free, W, N, table)[:2] == tuple(
        P.tables_reference(old, new, page, free, table, N)[:2])
    new = [0, 48, 17, 33]
    got = call_tables(None, new, page, free, W, N)
    want = P.tables_reference([0] * 4, new, page, free, [[0] * W] * 4, N)
    assert got == (want[0], want[1], [want[2]])


def test_no_slots_no_free_pages_and_pages_whose_slots_pass_32_bits():
    assert call_tables(None, [5, 0], 16, [], 2, 0) == ([[-1, -1], [-1, -1]], [[], []], [1])
    big = 2 ** 31 // 128                                   # the first slot of this page is 2^31
    t, s, n = call_tables(None, [2, 2], 128, [big, big - 1], 1, 2)
    assert t == [[big], [big - 1]] and n == [2]
    assert s == [[-1, -1], [2 ** 31 - 128, 2 ** 31 - 127]]


def pool(pages, page, heads, D, layout):
    shape = (pages, page, heads, D)
    k = torch.randn(shape, device="cuda").to(torch.bfloat16)
    v = torch.randn(shape, device="cuda").to(torch.bfloat16)
    if layout == "nhd":
        return k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    kv = torch.stack((k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)), 1).contiguous()
    return kv[:, 0], kv[:, 1]


@pytest.mark.parametrize("B,N,heads,D,page,layout,fused", [
    (1, 1, 1, 64, 16, "nhd", False), (1, 1, 8, 128, 16, "hnd", True), (64, 1, 8, 128, 16, "nhd", True),
    (3, 37, 5, 64, 32, "nhd", True), (2, 129, 3, 128, 128, "hnd", False), (4, 500, 16, 128, 64, "nhd", True),
    (7, 1001, 2, 64, 64, "hnd", True), (2, 9, 1, 128, 16, "nhd", False), (16, 700, 24, 128, 16, "nhd", False)])
def test_append_moves_every_named_row_and_no_other(B, N, heads, D, page, layout, fused):
    G.ensure_built()
    torch.manual_seed(B * N)
    r = random.Random(N)
    pages = -(-B * N // page) + 3
    ck, cv = pool(pages, page, heads, D, layout)
    if fused:                                              # views into one projection's output
        qkv = torch.randn((B, N, heads + 2 * heads, D), device="cuda").to(torch.bfloat16)
        k, v = (qkv[:, :, (1 + j) * heads:(2 + j) * heads].permute(0, 2, 1, 3) for j in range(2))
    else:
        k, v = (torch.randn((B, heads, N, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    all_slots = list(range(pages * page))
    r.shuffle(all_slots)
    slots = [[all_slots.pop() if r.random() < 0.9 else -1 - r.randrange(5) for _ in range(N)] for _ in range(B)]
    want_k, want_v = ck.clone(), cv.clone()
    live = [(b, i, s) for b, row in enumerate(slots) for i, s in enumerate(row) if s >= 0]
    if live:
        b, i, s = (torch.tensor(x, device="cuda") for x in zip(*live))
        want_k[s // page, :, s % page] = k[b, :, i]
        want_v[s // page, :, s % page] = v[b, :, i]
    cache = S.PageCache(ck, cv)
    wide = torch.full((B, N + 2), 2 ** 30, dtype=torch.int32, device="cuda")     # entries between rows are not slots
    wide[:, :N] = i32(slots)
    S.sage_cache_append(k, v, wide[:, :N], cache)
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(ck, want_k) and torch.equal(cv, want_v)


def test_a_slot_outside_the_cache_is_skipped_and_reported():
    G.ensure_built()
    ck, cv = pool(4, 16, 2, 64, "nhd")
    k, v = (torch.randn((1, 2, 3, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    want = ck.clone()
    want[1, :, 2] = k[0, :, 1]
    S.sage_cache_append(k, v, i32([[64, 18, 2 ** 31 - 1]]), S.PageCache(ck, cv))
    assert S.sage_get_device_status() == S.SAGE_ERR_PAGE
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(ck, want)


def test_append_behind_two_to_the_32_elements():
    """A cache of more than 2^32 elements: the last page's offsets pass 32 bits."""
    G.ensure_built()
    heads, D, page = 32, 128, 128
    pages = 2 ** 32 // (heads * D * page) + 3
    ck = torch.zeros((pages, page, heads, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    cv = torch.zeros((pages, page, heads, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    k, v = (torch.randn((1, heads, 2, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    S.sage_cache_append(k, v, i32([[pages * page - 1, (pages - 1) * page]]), S.PageCache(ck, cv))
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    for c, x in ((ck, k), (cv, v)):
        assert torch.equal(c[-1, :, -1], x[0, :, 0]) and torch.equal(c[-1, :, 0], x[0, :, 1])
        assert int(c.permute(0, 2, 1, 3)[:-1].count_nonzero()) == 0
