"""Attention of a tree of drafted tokens over a page cache against its
definition in 64 bits.  Cache rows that no length covers are NaN and unused
table entries lie outside the cache, so reading either shows."""
import random

import pytest
import torch

import quantized_exact_attention_gb300 as S
from tests import gpu_support as G
from tests import paged_support as P
from tests import tree_support as T

pytestmark = pytest.mark.gpu

# A wide table (its entries behind the lengths unused) takes the list, a narrow one whole items.
wide = pytest.mark.parametrize("wide", [0, 1])


def pad(on):
    return {"table_pad": 1200 if on else 2}


def trees(B, N, deep, seed):
    r = random.Random(seed)
    return [T.sees_of(T.random_parents(r, N, deep)) for _ in range(B)]


def anything(B, N, seed):
    """Masks that are no trees: tokens that see later ones, or nothing."""
    r = random.Random(seed)
    return [[{t for t in range(N) if r.random() < 0.4} if r.random() < 0.8 else set() for _ in range(N)] for _ in range(B)]


def mask_of(sees, N, width=None):
    return T.i32([T.words_of(s, N, width) for s in sees])


def go(sees, **kw):
    G.ensure_built()
    p = P.make(causal=False, **kw)
    T.check(p, sees, T.run(p, mask_of(sees, kw["Nq"])))
    return p


@wide
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Nq,H,Hkv", [(1, 2, 2), (3, 2, 2), (8, 8, 8), (5, 6, 2), (16, 1, 1), (2, 16, 2), (17, 2, 2), (26, 8, 2),
                                      (64, 2, 1), (33, 24, 8), (130, 2, 1), (260, 3, 3)])
def test_shapes(Nq, H, Hkv, D, wide):
    B = 4
    kv = [Nq, Nq + 100, Nq + 1, Nq + 37]
    go(trees(B, Nq, 5, Nq), B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=32, kv_len=kv, q_len=[Nq, max(1, Nq // 2), Nq - 1, Nq],
       seed=Nq, **pad(wide))


@wide
@pytest.mark.parametrize("Nq", [1, 7, 16, 31, 32, 33, 64, 65, 96, 128, 200])
@pytest.mark.parametrize("base", [0, 1, 15, 63, 64, 100, 127, 128, 129])
def test_where_the_new_tokens_begin(Nq, base, wide):
    """The mask's window at every kind of place in a tile and in a half of one."""
    go(trees(2, Nq, 9, base), B=2, H=2, Hkv=2, D=64, Nq=Nq, page=16, kv_len=[base + Nq, base + Nq], seed=base, **pad(wide))


@wide
@pytest.mark.parametrize("Nq,G", [(6, 2), (20, 1), (70, 4), (150, 1)])
@pytest.mark.parametrize("prefix", [0, 50])
def test_masks_that_are_no_trees(Nq, G, prefix, wide):
    """Later tokens, no token at all; rows that see nothing are zero.  Fewer keys than query rows, none, no rows."""
    B = 6
    sees = anything(B, Nq, Nq)
    p = go(sees, B=B, H=2 * G, Hkv=2, D=128, Nq=Nq, page=16, q_len=[Nq, Nq, Nq, Nq - 1, 0, Nq],
           kv_len=[Nq, Nq + 40, max(Nq - 3, 0), Nq - 1, 5, 0], prefix=prefix, seed=Nq, **pad(wide))
    if prefix == 0:
        o = T.run(p, mask_of(sees, Nq))
        torch.cuda.synchronize()
        for i in (i for i in range(Nq) if not sees[0][i]):
            assert int(o[0, :, i].count_nonzero()) == 0
        assert int(o[5].count_nonzero()) == 0


@pytest.mark.parametrize("B,Hkv,G,Nq,D,prefix", [
    (40, 8, 1, 1, 128, 1700), (33, 8, 2, 3, 128, 2100), (300, 2, 4, 2, 64, 2000),      # few rows beside the prefix's list
    (24, 4, 4, 13, 64, 4099), (32, 4, 4, 5, 64, 4099), (3, 1, 1, 17, 128, 1000), (9, 8, 4, 5, 128, 4099),
    (4, 2, 4, 40, 128, 300)])
def test_shared_prefix(B, Hkv, G, Nq, D, prefix):
    kv = [(37 * b) % 90 for b in range(B)]
    q = [min(Nq, 1 + b % Nq) if b % 7 else 0 for b in range(B)]
    go(trees(B, Nq, 3, B), B=B, H=Hkv * G, Hkv=Hkv, D=D, Nq=Nq, page=32, kv_len=kv, q_len=q, prefix=prefix, seed=prefix + B)


@wide
@pytest.mark.parametrize("G", [100, 128, 129, 300])
@pytest.mark.parametrize("Nq", [1, 3, 40])
def test_many_heads_to_a_key_head(G, Nq, wide):
    """Over 128: the few-rows kernel, also for more than 32 tokens."""
    go(trees(2, Nq, 4, G), B=2, H=G, Hkv=1, D=64, Nq=Nq, page=16, kv_len=[Nq + 77, Nq], q_len=[Nq, max(1, Nq - 1)], seed=G,
       **pad(wide))


# Lists: two lanes a row (up to 64 rows of 64 channels) with whole and cut items, few items of many parts, and others.
@pytest.mark.parametrize("B,H,Hkv,Nq,n,D", [
    (150, 4, 2, 12, 500, 64), (40, 32, 8, 16, 900, 64), (1, 2, 1, 32, 30000, 64), (3, 8, 2, 16, 9000, 64), (2, 4, 2, 20, 20000, 128),
    (1, 6, 2, 100, 15000, 128), (1, 4, 4, 40, 12000, 64)])
@pytest.mark.parametrize("page", [16, 128])
def test_lists(B, H, Hkv, Nq, n, D, page):
    kv = [max(0, n - 397 * b % (n + 1)) for b in range(B)]
    q = [Nq if b % 4 else max(0, Nq - 3 * b % (Nq + 1)) for b in range(B)]
    sees = trees(1, Nq, 3, n) * B
    p = go(sees, B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=page, q_len=q, kv_len=kv, seed=n, table_pad=3000 // page)
    first = T.run(p, mask_of(sees, Nq))
    assert all(torch.equal(first, T.run(p, mask_of(sees, Nq))) for _ in range(3))


@pytest.mark.parametrize("B,H,Hkv,Nq,n,D", [(1, 8, 8, 8, 777, 128), (32, 32, 8, 26, 3000, 128), (4, 24, 8, 251, 5000, 128),
                                            (50, 32, 8, 32, 500, 128), (3, 6, 3, 500, 1100, 64), (1, 8, 2, 64, 40000, 128)])
def test_long_sequences(B, H, Hkv, Nq, n, D):
    kv = [max(Nq, n - 211 * b % n) for b in range(B)]
    go(trees(B, Nq, 12, n), B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=64, kv_len=kv, seed=n, table_pad=0)


# Items that clusters of 1 to 8 CTAs take whole: up to 64 rows (two lanes each), to 128, and several sets of rows;
# requests much shorter than the table is wide, without keys and without rows.
@pytest.mark.parametrize("B,H,Hkv,Nq,n,D", [
    (1, 4, 1, 16, 3000, 64), (1, 8, 8, 9, 900, 128), (3, 24, 12, 20, 1200, 64), (5, 32, 8, 13, 800, 128), (6, 16, 8, 5, 1500, 64),
    (16, 8, 4, 32, 1000, 128), (70, 1, 1, 60, 2000, 64), (24, 16, 4, 4, 2500, 128), (36, 8, 4, 16, 1500, 64),
    (140, 2, 1, 40, 1400, 64), (140, 2, 1, 40, 1400, 128), (270, 2, 1, 7, 1000, 64), (36, 4, 4, 2, 1600, 64), (47, 6, 2, 3, 900, 64),
    (2, 32, 8, 26, 5000, 64), (9, 32, 8, 26, 900, 128), (2, 16, 2, 100, 2000, 128), (1, 8, 4, 250, 4000, 64), (1, 100, 1, 7, 1100, 64),
    (3, 66, 2, 1, 1500, 64), (2, 64, 1, 1, 1800, 128), (9, 64, 2, 2, 1000, 128)])
@pytest.mark.parametrize("prefix", [0, 700])
def test_clusters(B, H, Hkv, Nq, n, D, prefix):
    kv = [max(0, n - 397 * b % (n + 1)) for b in range(B)]
    q = [Nq if b % 4 else max(0, Nq - 3 * b % (Nq + 1)) for b in range(B)]
    kv[-1], q[0] = (kv[-1], Nq) if B == 1 else (0, Nq)
    kv[0] = n
    deep = 3 if B < 100 else 0
    sees = trees(1, Nq, deep, n) * B if B > 20 else trees(B, Nq, deep, n)
    go(sees, B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=(16, 64, 128)[B % 3], q_len=q, kv_len=kv, prefix=prefix, seed=n, table_pad=0)


def test_layouts_scale_and_shared_masks():
    G.ensure_built()
    B, Nq = 3, 21
    sees = trees(1, Nq, 4, 3) * B
    for layout in ("nhd", "hnd"):
        p = P.make(B=B, H=8, Hkv=2, D=64, Nq=Nq, page=16, kv_len=[60, 21, 200], layout=layout, causal=False, sm_scale=0.31)
        for mask in (mask_of(sees[:1], Nq)[0], mask_of(sees, Nq, 4), mask_of(sees[:1], Nq).expand(B, Nq, 1),
                     torch.stack((mask_of(sees, Nq, 2), mask_of(sees, Nq, 2)), 2)[:, :, 1]):
            T.check(p, sees, T.run(p, mask))


@wide
@pytest.mark.parametrize("Nq,G", [(1, 1), (5, 2), (30, 4), (200, 1)])
def test_where_all_is_seen(Nq, G, wide):
    """All bits set: attention without a mask; bits and rows behind q_len do not matter, to the last bit."""
    p = P.make(B=3, H=2 * G, Hkv=2, D=128, Nq=Nq, page=32, q_len=[Nq, max(1, Nq - 2), Nq], kv_len=[Nq + 50, Nq, 700],
               causal=False, **pad(wide))
    ones = torch.full((3, Nq, -(-Nq // 32)), -1, dtype=torch.int32, device="cuda")
    o = T.run(p, ones)
    P.check(p, o)
    exact = mask_of([[set(range(n))] * n + [set()] * (Nq - n) for n in p.q_len], Nq)
    assert torch.equal(T.run(p, exact), o)


def test_chain_is_the_causal_mask():
    G.ensure_built()
    for Nq in (4, 40, 300):
        p = P.make(B=2, H=4, Hkv=2, D=64, Nq=Nq, page=16, kv_len=[Nq + 30, Nq], causal=True)
        mask, depth = S.tree_tables(T.i32([list(range(-1, Nq - 1))] * 2))
        P.check(p, T.run(p, mask))
        assert depth[0].tolist() == list(range(Nq))


@pytest.mark.parametrize("pages,far", [(40, 50), (100, 350), (1300, 400)])     # an item a CTA, a cluster, the list
def test_streams_graphs_and_repeats(pages, far):
    """Two calls in flight on their own streams and workspaces; a captured call that serves later lengths, masks and
    tables; equal bits for equal inputs."""
    G.ensure_built()
    B, Nq = 5, 18
    ps = [P.make(B=B, H=8, Hkv=2, D=128, Nq=Nq, page=16, kv_len=[Nq + far * b + s for b in range(B)], causal=False, seed=s,
                 table_pad=pages - (Nq + 4 * far + s + 15) // 16) for s in range(2)]
    sees = [trees(B, Nq, 3, s) for s in range(2)]
    masks = [mask_of(s, Nq) for s in sees]
    want = [T.run(p, m) for p, m in zip(ps, masks)]
    for p, s, o in zip(ps, sees, want):
        T.check(p, s, o)
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [torch.full_like(o, 7.0) for o in want]
    ws = [S.alloc_paged_workspace(B, 8, 2, Nq, 128) for _ in ps]
    torch.cuda.synchronize()
    for _ in range(4):
        for p, m, o, w, st in zip(ps, masks, outs, ws, streams):
            with torch.cuda.stream(st):
                T.run(p, m, workspace=w, o=o)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # one graph, its buffers filled anew
    cache = S.PageCache(ps[0].cache_k, ps[0].cache_v)
    q, mask, table, kv, o = ps[0].q.clone(), masks[0].clone(), ps[0].table.clone(), T.i32(ps[0].kv_len), torch.zeros_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.sage_attn_paged_tree(q, o, cache, table, mask, ws[0], kv_len=kv)
    for n in (0, 3, 11):
        new = trees(B, Nq, 3, 50 + n)
        p = P.Paged(ps[0].q.flip(0), ps[0].cache_k, ps[0].cache_v, ps[0].table, [Nq] * B, [x - n for x in ps[0].kv_len], None,
                    0, False)
        p.kv_len = [max(x, 1) for x in p.kv_len]
        q.copy_(p.q)
        mask.copy_(mask_of(new, Nq))
        kv.copy_(T.i32(p.kv_len))
        graph.replay()
        T.check(p, new, o)


def test_an_unlisted_page_is_recorded():
    G.ensure_built()
    for Nq in (2, 40):
        p = P.make(B=1, H=2, Hkv=2, D=64, Nq=Nq, page=16, kv_len=[Nq + 20], causal=False)
        p.table[0, 0] = 1000
        o = T.run(p, mask_of(trees(1, Nq, 3, 1), Nq))
        assert S.sage_get_device_status() == S.SAGE_ERR_PAGE
        assert S.sage_get_device_status() == S.SAGE_OK
        assert bool(torch.isfinite(o).all())


def test_a_withheld_copy_runs_out():
    """The bounded waits of every form of the many-rows kernel: the call ends, says so, and the next one is right."""
    G.ensure_built()
    for D, Nq, n, list_ in ((128, 40, 100, 0), (64, 40, 100, 1), (64, 20, 100, 1), (128, 20, 900, 0), (64, 20, 900, 0), (128, 100, 900, 0)):
        p = P.make(B=1, H=2, Hkv=1, D=D, Nq=Nq, page=64, kv_len=[Nq + n], seed=D, causal=False, **pad(list_))
        sees = trees(1, Nq, 3, D)
        S.sage_debug_inject_fault(1)
        T.run(p, mask_of(sees, Nq))
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_ERR_TIMEOUT
        T.check(p, sees, T.run(p, mask_of(sees, Nq)))


def test_cache_offsets_behind_two_to_the_32_elements():
    G.ensure_built()
    heads, D, page = 32, 128, 128
    pages = 2 ** 32 // (heads * D * page) + 4
    k = torch.zeros((pages, page, heads, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    v = torch.zeros((pages, page, heads, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    g = torch.Generator(device="cuda").manual_seed(5)
    last = torch.tensor([[pages - 1, pages - 3, pages - 2, 0, pages - 4, 5, 7]], dtype=torch.int32, device="cuda")
    for pg in last.unique().tolist():
        k[pg] = torch.randn((heads, page, D), device="cuda", generator=g).to(torch.bfloat16)
        v[pg] = torch.randn((heads, page, D), device="cuda", generator=g).to(torch.bfloat16)
    for Nq, n, width in ((3, 300, 3), (20, 300, 3), (20, 850, 7)):
        q = torch.randn((1, heads, Nq, D), device="cuda", generator=g).to(torch.bfloat16)
        sees = trees(1, Nq, 3, Nq)
        p = P.Paged(q, k, v, last[:, :width].contiguous(), [Nq], [n], None, 0, False)
        T.check(p, sees, T.run(p, mask_of(sees, Nq)))
    # rows of the append and of the move there
    from_, to = (pages - 1) * page + 5, (pages - 2) * page + 100
    r = S.make_rotary(S.rotary_frequencies(D)[0])
    new = torch.randn((1, heads, 1, D), device="cuda", generator=g).to(torch.bfloat16)
    S.sage_cache_append_rope(new, new, T.i32([[from_]]), S.PageCache(k, v), r, start=T.i32([77]))
    S.sage_cache_keep(T.i32([[1]]), T.i32([[to, from_]]), S.PageCache(k, v))
    turned = S.rope(new, r, start=T.i32([77]))
    torch.cuda.synchronize()
    for pg, off in ((pages - 1, 5), (pages - 2, 100)):
        assert torch.equal(k[pg, :, off], turned[0, :, 0]) and torch.equal(v[pg, :, off], new[0, :, 0])


def test_refusals_of_the_binding():
    G.ensure_built()
    p = P.make(B=2, H=2, Hkv=2, D=64, Nq=40, page=16, kv_len=[50, 60], causal=False)
    good = mask_of(trees(2, 40, 3, 1), 40)
    for bad in (good[:, :39], good[:1], good[..., :1], good.float(), good.transpose(1, 2), good[0, 0], good.cpu()):
        with pytest.raises(ValueError):
            T.run(p, bad)


# Which form a call takes, by the widths of its tables in tiles of 128 keys: one launch where clusters or CTAs take whole
# items, two from a list with its join, three where the prefix has a list of its own besides.  Both sides of each bound.
@pytest.mark.parametrize("B,H,Hkv,D,Nq,own,pre,launches", [
    (24, 16, 4, 64, 13, 36, 0, 1), (24, 16, 4, 64, 13, 37, 0, 2),                     # 12 tiles a CTA of clusters of 3
    (24, 16, 4, 128, 13, 36, 0, 1), (24, 16, 4, 128, 13, 37, 0, 2),
    (24, 16, 4, 64, 13, 8, 42, 1), (24, 16, 4, 64, 13, 8, 43, 2),                     # 64 channels: a prefix's count 2 / 3
    (24, 16, 4, 128, 13, 8, 28, 1), (24, 16, 4, 128, 13, 8, 29, 2), (24, 16, 4, 128, 13, 8, 42, 2),        # 128: whole
    (24, 16, 4, 64, 13, 64, 33, 2),                        # a table far wider than its requests
    (1, 4, 1, 64, 16, 35, 0, 1), (1, 4, 1, 64, 16, 36, 0, 2),                         # few key sequences
    (1, 4, 1, 128, 4, 52, 0, 1), (1, 4, 1, 128, 4, 53, 0, 2),                         # ... of up to 16 rows
    (2, 16, 2, 128, 100, 24, 0, 1), (2, 16, 2, 128, 100, 45, 0, 2),                   # several sets of rows
    (6, 16, 8, 64, 5, 12, 0, 1), (150, 4, 2, 64, 12, 200, 0, 2), (3, 6, 3, 64, 500, 48, 0, 1), (3, 6, 3, 64, 500, 49, 0, 2),
    (16, 8, 8, 128, 4, 2, 33, 3), (2, 4, 2, 128, 40, 1, 0, 1)])
def test_which_form_a_call_takes(B, H, Hkv, D, Nq, own, pre, launches):
    G.ensure_built()
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the bounds are those of 152 SMs")
    page = 128
    p = P.make(B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=page, kv_len=[min(own * page, Nq + 50 * (b % 4)) for b in range(B)],
               prefix=300 if pre else 0, causal=False, seed=own, table_pad=0)

    def widened(t, width):
        return torch.cat((t, t.new_full(t.shape[:-1] + (width - t.shape[-1],), p.cache_k.shape[0] + 9)), -1)

    p.table = widened(p.table, own)
    if pre:
        p.prefix_table = widened(p.prefix_table, pre)
    sees = trees(1, Nq, 3, own) * B
    o = T.run(p, mask_of(sees, Nq))
    assert S.sage_last_launch_count() == launches
    T.check(p, sees, o)
