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


@pytest.mark.parametrize("B,H,Hkv,Nq,n,D", [(1, 8, 8, 8, 777, 128), (32, 32, 8, 26, 3000, 128), (4, 24, 8, 251, 5000, 128),
                                            (50, 32, 8, 32, 500, 128), (3, 6, 3, 500, 1100, 64), (1, 8, 2, 64, 40000, 128)])
def test_long_sequences(B, H, Hkv, Nq, n, D):
    kv = [max(Nq, n - 211 * b % n) for b in range(B)]
    go(trees(B, Nq, 12, n), B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=64, kv_len=kv, seed=n, table_pad=0)


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
def test_equal_to_the_unmasked_form_where_all_is_seen(Nq, G, wide):
    """All bits set: the same arithmetic as sage_attn_paged without a causal mask, bit for bit; bits and rows behind
    q_len do not matter."""
    _ = wide
    p = P.make(B=3, H=2 * G, Hkv=2, D=128, Nq=Nq, page=32, q_len=[Nq, max(1, Nq - 2), Nq], kv_len=[Nq + 50, Nq, 700],
               causal=False, **pad(wide))
    want = P.run(p)
    ones = torch.full((3, Nq, -(-Nq // 32)), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(T.run(p, ones), want)
    exact = mask_of([[set(range(n))] * n + [set()] * (Nq - n) for n in p.q_len], Nq)
    assert torch.equal(T.run(p, exact), want)


def test_chain_is_the_causal_mask():
    G.ensure_built()
    for Nq in (4, 40, 300):
        p = P.make(B=2, H=4, Hkv=2, D=64, Nq=Nq, page=16, kv_len=[Nq + 30, Nq], causal=True)
        mask, depth = S.tree_tables(T.i32([list(range(-1, Nq - 1))] * 2))
        P.check(p, T.run(p, mask))
        assert depth[0].tolist() == list(range(Nq))


def test_streams_graphs_and_repeats():
    """Two calls in flight on their own streams and workspaces; a captured call that serves later lengths, masks and
    tables; equal bits for equal inputs."""
    G.ensure_built()
    B, Nq = 5, 18
    ps = [P.make(B=B, H=8, Hkv=2, D=128, Nq=Nq, page=16, kv_len=[Nq + 50 * b + s for b in range(B)], causal=False, seed=s,
                 table_pad=40 - (Nq + 200 + s + 15) // 16) for s in range(2)]
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


def test_refusals_of_the_binding():
    G.ensure_built()
    p = P.make(B=2, H=2, Hkv=2, D=64, Nq=40, page=16, kv_len=[50, 60], causal=False)
    good = mask_of(trees(2, 40, 3, 1), 40)
    for bad in (good[:, :39], good[:1], good[..., :1], good.float(), good.transpose(1, 2), good[0, 0], good.cpu()):
        with pytest.raises(ValueError):
            T.run(p, bad)
