"""Tree tables and the move of accepted tokens, against their definition."""
import random

import pytest
import torch

import quantized_exact_attention_gb300 as S
from tests import gpu_support as G
from tests import tree_support as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 2, 7, 31, 32, 33, 64, 65, 100, 127, 128, 129, 250, 256, 257, 513, 1000])
@pytest.mark.parametrize("B,deep", [(1, 3), (5, 0), (37, 40)])
def test_tables(B, N, deep):
    G.ensure_built()
    r = random.Random(N + B)
    parents = [T.random_parents(r, N, deep) for _ in range(B)]
    n_len = [r.choice((N, N, 0, 1, -4, N + 7, r.randrange(N + 1))) for _ in range(B)]
    for lens in (None, n_len):
        mask, depth = S.tree_tables(T.i32(parents), T.i32(lens) if lens else None)
        torch.cuda.synchronize()
        for b in range(B):
            n = N if lens is None else min(max(lens[b], 0), N)
            sees = T.sees_of(parents[b])[:n] + [set()] * (N - n)
            assert mask[b].tolist() == T.words_of(sees, N)
            assert depth[b].tolist() == [max(len(s) - 1, 0) for s in sees]


def test_the_largest_tree():
    G.ensure_built()
    r = random.Random(5)
    parents = [T.random_parents(r, 4096, 900), T.random_parents(r, 4096, 0)]
    mask, depth = S.tree_tables(T.i32(parents))
    for b in range(2):
        sees = T.sees_of(parents[b])
        assert depth[b].tolist() == [len(s) - 1 for s in sees]
        for i in (0, 1, 31, 32, 2047, 4000, 4095):
            assert mask[b, i].tolist() == T.words_of([sees[i]], 4096)[0]


def test_parents_that_are_none():
    """Negative numbers, the token itself and those behind it: no parent."""
    G.ensure_built()
    parents = [[5, -1, 1, 3, 2, 2 ** 31 - 1, -2 ** 31, 6]]
    mask, depth = S.tree_tables(T.i32(parents))
    sees = T.sees_of(parents[0])
    assert sees[2] == {1, 2} and sees[3] == {3} and sees[5] == {5} and sees[7] == {6, 7}
    assert mask[0].tolist() == T.words_of(sees, 8) and depth[0].tolist() == [0, 0, 1, 0, 2, 0, 0, 1]


@pytest.mark.parametrize("N", [5, 40, 300])
def test_tables_into_strided_tensors(N):
    """Wider rows, rows apart, no depth: what lies between is left as it is."""
    G.ensure_built()
    B, W = 3, -(-N // 32)
    r = random.Random(N)
    parents = [T.random_parents(r, N, 6) for _ in range(B)]
    p = T.i32([row + [9] * 4 for row in parents])[:, :N]
    mask = torch.full((B, N + 2, W + 3), 77, dtype=torch.int32, device="cuda")
    depth = torch.full((B, N + 5), 77, dtype=torch.int32, device="cuda")
    S.sage_tree_tables(p, mask[:, :N], depth[:, :N])
    S.sage_tree_tables(p, mask[:, :N])
    torch.cuda.synchronize()
    for b in range(B):
        sees = T.sees_of(parents[b])
        assert mask[b, :N, :W].tolist() == T.words_of(sees, N)
        assert depth[b, :N].tolist() == [len(s) - 1 for s in sees]
    assert bool((mask[:, N:] == 77).all()) and bool((mask[:, :, W:] == 77).all()) and bool((depth[:, N:] == 77).all())
    first = torch.zeros((B, N, W), dtype=torch.int32, device="cuda")
    S.sage_tree_tables(T.i32(parents[0])[None].expand(B, N), first)            # one tree for all requests
    assert all(first[b].tolist() == T.words_of(T.sees_of(parents[0]), N) for b in range(B))


# ---------------------------------------------------------------------------
def moved(kept, slots, cache):
    """cache.k and cache.v after the moves, from the definition."""
    page = cache.page_size
    out = []
    for t in (cache.k, cache.v):
        rows = t.permute(0, 2, 1, 3).reshape(-1, t.shape[1], t.shape[3]).clone()
        where = T.keep_reference(kept, slots, {s: s for row in slots for s in row if s >= 0})
        src = torch.tensor(list(where.values()), device="cuda", dtype=torch.long)
        dst = torch.tensor(list(where.keys()), device="cuda", dtype=torch.long)
        if len(where):
            rows[dst] = rows[src].clone()
        out.append(rows.reshape(t.shape[0], page, t.shape[1], t.shape[3]).permute(0, 2, 1, 3))
    return out


def fresh(n_pages, page, H, D, layout, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (n_pages, page, H, D) if layout == "nhd" else (n_pages, H, page, D)
    t = [torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    return S.PageCache(*(x.permute(0, 2, 1, 3) if layout == "nhd" else x for x in t))


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("B,H,D,page,N,K", [(1, 1, 64, 16, 1, 1), (64, 8, 128, 16, 26, 6), (7, 3, 64, 32, 40, 40),
                                            (5, 2, 128, 64, 100, 70), (3, 16, 128, 128, 9, 8), (2, 5, 64, 16, 300, 33),
                                            (700, 2, 64, 16, 20, 12), (2, 40, 128, 64, 80, 64)])
def test_keep_accepted_paths(B, H, D, page, N, K, layout):
    """Paths of random trees: moves to the front, whose sources may be destinations of others."""
    G.ensure_built()
    r = random.Random(N + K)
    cache = fresh(B * -(-N // page) + 2, page, H, D, layout)
    order = torch.randperm(cache.num_pages * page, generator=torch.Generator().manual_seed(K))[:B * N].reshape(B, N).tolist()
    kept = []
    for _ in range(B):
        path = sorted(r.sample(range(N), r.randint(0, K)))
        kept.append(path + [-1] * (K - len(path)))
    want = moved(kept, order, cache)
    S.sage_cache_keep(T.i32(kept), T.i32(order), cache)
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(cache.k, want[0]) and torch.equal(cache.v, want[1])


@pytest.mark.parametrize("B", [6, 650])                   # several groups of threads to a block, and one
@pytest.mark.parametrize("N,K", [(4, 4), (9, 8), (33, 33), (80, 64), (100, 97)])
def test_keep_in_any_order(N, K, B):
    """Entries in any order, repeated, out of range, and tokens without a place: one move after another."""
    G.ensure_built()
    page = 16
    r = random.Random(N)
    cache = fresh(B * -(-N // page) + 2, page, 2, 64, "nhd")
    order = torch.randperm(cache.num_pages * page, generator=torch.Generator().manual_seed(K))[:B * N].reshape(B, N).tolist()
    for row in order:
        for i in range(N):
            if r.random() < 0.2:
                row[i] = -r.randrange(1, 9)
    kept = [[r.choice((r.randrange(N), r.randrange(N), -1, N, -7, 2 ** 31 - 1)) for _ in range(K)] for _ in range(B)]
    kept[0] = list(range(K))                               # nothing moves
    kept[1] = [min(i + 1, N - 1) for i in range(K)]        # each from the place behind
    kept[2] = [max(i - 1, 0) for i in range(K)]            # the first, handed on from place to place
    want = moved(kept, order, cache)
    S.sage_cache_keep(T.i32(kept), T.i32(order), cache)
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(cache.k, want[0]) and torch.equal(cache.v, want[1])


def test_keep_outside_the_cache_is_recorded():
    G.ensure_built()
    cache = fresh(4, 16, 2, 128, "nhd")
    slots, kept = [[1, 64, 3, 4], [2 ** 31 - 1, 9, 10, 11]], [[2, 3, 1], [3, 0, 3]]
    # request 0: 3 -> 1, (4 -> 64: outside), (64 -> 3: outside); request 1: (11 -> outside), (outside -> 9), 11 -> 10
    k, v = cache.k.clone(), cache.v.clone()
    for t in (k, v):
        rows = t.permute(0, 2, 1, 3)
        rows[0, 1], rows[0, 10] = rows[0, 3].clone(), rows[0, 11].clone()
    S.sage_cache_keep(T.i32(kept), T.i32(slots), cache)
    assert S.sage_get_device_status() == S.SAGE_ERR_PAGE
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)


@pytest.mark.parametrize("B,K", [(300, 6), (300, 8), (400, 8), (400, 10), (400, 11), (400, 33), (600, 12), (700, 12), (700, 40)])
def test_keep_on_all_sides_of_its_rule(B, K):
    """Up to two, four and more blocks an SM (a block for each request here), few entries and many: paths and any order."""
    G.ensure_built()
    page, N = 16, K + 9
    r = random.Random(B + K)
    cache = fresh(B * -(-N // page) + 2, page, 3, 64, "nhd")
    order = torch.randperm(cache.num_pages * page, generator=torch.Generator().manual_seed(K))[:B * N].reshape(B, N).tolist()
    kept = []
    for b in range(B):
        path = sorted(r.sample(range(N), r.randint(0, K))) if b % 3 else [r.randrange(-2, N + 1) for _ in range(K)]
        kept.append(path + [-1] * (K - len(path)))
    want = moved(kept, order, cache)
    S.sage_cache_keep(T.i32(kept), T.i32(order), cache)
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(cache.k, want[0]) and torch.equal(cache.v, want[1])
