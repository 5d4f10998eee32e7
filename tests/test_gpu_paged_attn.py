"""Attention over a page cache against its definition in 64 bits.  Rows of the
cache that no length covers are NaN and unused table entries lie outside the
cache, so reading either shows."""
import pytest
import torch

import quantized_exact_attention_gb300 as S
from tests import gpu_support as G
from tests import paged_support as P

pytestmark = pytest.mark.gpu


def go(**kw):
    G.ensure_built()
    p = P.make(**kw)
    P.check(p, P.run(p))
    return p


# Few rows: a wide table (its entries behind the lengths unused) takes the list,
# a narrow one clusters that each take an item whole.
wide = pytest.mark.parametrize("wide", [0, 1])


def pad(wide):
    return {"table_pad": 1200 if wide else 2}


@wide
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500])
def test_one_token_one_request(D, page, n, wide):
    go(B=1, H=2, Hkv=2, D=D, Nq=1, page=page, kv_len=[n], seed=n, **pad(wide))


@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,n", [(1, 180), (1, 300), (1, 1000), (3, 2000), (9, 700), (36, 700), (37, 350), (75, 190), (77, 190)])
def test_sequences_of_one_cluster(B, n, G, D):
    """From one CTA to clusters of eight, up to the shares where the list takes over."""
    go(B=B, H=8 * G, Hkv=8, D=D, Nq=1, page=16, kv_len=[max(0, n - 37 * b % (n + 1)) for b in range(B)], table_pad=0, seed=n)


@wide
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (6, 2), (8, 1), (24, 8), (16, 1), (9, 3), (20, 1), (33, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(H, Hkv, D, wide):
    go(B=3, H=H, Hkv=Hkv, D=D, Nq=1, page=16, kv_len=[70, 1, 333], seed=H, **pad(wide))


@wide
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Nq,G", [(2, 1), (5, 2), (3, 8), (17, 3), (40, 1), (129, 2)])
def test_several_tokens(layout, causal, Nq, G, wide):
    kv = [Nq, Nq + 100, Nq + 1, Nq + 37]
    go(B=4, H=2 * G, Hkv=2, D=128, Nq=Nq, page=32, kv_len=kv, q_len=[Nq, 1, Nq - 1, Nq], causal=causal, layout=layout,
       seed=Nq, **pad(wide))


@pytest.mark.parametrize("B,H,Hkv,Nq,n,D", [
    (25, 8, 8, 300, 300, 128), (40, 8, 8, 150, 700, 64), (50, 32, 8, 32, 500, 128), (90, 24, 8, 20, 1500, 64),
    (3, 6, 3, 700, 1100, 128), (38, 8, 8, 100, 130, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_items_taken_whole(B, H, Hkv, Nq, n, D, causal):
    """More items than CTAs at a time, and fewer; requests of very different lengths."""
    kv = [max(Nq if b % 3 else 0, n - 211 * b % n) for b in range(B)]
    q = [Nq - 17 * b % (Nq + 1) for b in range(B)]
    go(B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=64, q_len=q, kv_len=kv, causal=causal, table_pad=0, seed=n)


# A key head with so many query heads that a group of 128 rows holds one token,
# or (over 128) not a whole one.
@wide
@pytest.mark.parametrize("G,Hkv", [(65, 2), (100, 1), (128, 2), (129, 1), (150, 2), (300, 1)])
@pytest.mark.parametrize("Nq,causal", [(1, True), (3, True), (3, False), (9, True)])
@pytest.mark.parametrize("prefix", [0, 130])
def test_many_heads_to_a_key_head(G, Hkv, Nq, causal, prefix, wide):
    kv = [0, Nq, 1, 300, 77]
    go(B=5, H=G * Hkv, Hkv=Hkv, D=64, Nq=Nq, page=16, kv_len=kv, q_len=[Nq, Nq, Nq, 0, max(1, Nq - 1)], prefix=prefix,
       causal=causal, seed=G + Nq, **pad(wide))


@wide
@pytest.mark.parametrize("prefix", [1, 16, 100, 128, 777])
@pytest.mark.parametrize("B,Nq,G", [(1, 1, 1), (3, 1, 2), (5, 1, 8), (20, 1, 4), (4, 3, 2), (2, 30, 2), (70, 1, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_shared_prefix(prefix, B, Nq, G, D, wide):
    kv = [Nq + (37 * b) % 90 for b in range(B)]
    go(B=B, H=2 * G, Hkv=2, D=D, Nq=Nq, page=16, kv_len=kv, prefix=prefix, seed=prefix + B,
       **pad(wide))


# A prefix whose repeated reading would cost over 134 MB is read once for all
# rows: few rows, one and two groups of 128 rows, a last group that is not full.
@pytest.mark.parametrize("B,Hkv,G,Nq,D,prefix", [
    (40, 8, 1, 1, 128, 1700), (70, 4, 8, 1, 64, 4001), (33, 8, 2, 3, 128, 2100), (300, 2, 4, 2, 64, 2000),
    (8, 16, 16, 1, 64, 8200), (2, 8, 3, 5, 128, 33000), (129, 8, 1, 1, 64, 1025), (17, 4, 5, 3, 128, 8000)])
def test_long_shared_prefix(B, Hkv, G, Nq, D, prefix):
    kv = [(37 * b) % 90 for b in range(B)]
    q = [min(Nq, 1 + b % Nq) if b % 7 else 0 for b in range(B)]
    go(B=B, H=Hkv * G, Hkv=Hkv, D=D, Nq=Nq, page=32, kv_len=kv, q_len=q, prefix=prefix, seed=prefix + B)


# Between 17 and 64 rows to a key head: with enough to save, the prefix's items
# and the requests' in one list; short and long prefixes, prefixes of which the
# device says less than its table lists, requests without rows or keys.
@pytest.mark.parametrize("B,Hkv,G,Nq,D", [
    (2, 1, 17, 1, 64), (3, 1, 1, 17, 128), (32, 4, 4, 5, 64), (9, 8, 4, 5, 128), (7, 3, 8, 8, 128), (65, 2, 8, 3, 64),
    (130, 1, 64, 1, 128), (40, 2, 1, 33, 64), (300, 3, 9, 7, 64)])
@pytest.mark.parametrize("prefix", [1, 130, 1000, 4099])
@pytest.mark.parametrize("causal", [True, False])
def test_prefix_for_some_rows(B, Hkv, G, Nq, D, prefix, causal):
    kv = [(37 * b) % 300 if b % 5 else 0 for b in range(B)]
    q = [min(Nq, 1 + b % (Nq + 3)) if b % 7 else 0 for b in range(B)]
    p = go(B=B, H=Hkv * G, Hkv=Hkv, D=D, Nq=Nq, page=32, kv_len=kv, q_len=q, prefix=prefix, causal=causal,
           seed=prefix + B)
    for p.prefix_len in (prefix // 3, 0):
        P.check(p, P.run(p))


@wide
@pytest.mark.parametrize("prefix", [0, 50])
@pytest.mark.parametrize("Nq", [1, 4, 40])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_without_keys(prefix, Nq, causal, wide):
    """No own keys, no query rows, and (causal) fewer keys than query rows: rows that see nothing are zero."""
    p = go(B=5, H=4, Hkv=2, D=64, Nq=Nq, page=16, q_len=[Nq, 0, Nq, Nq, 0], kv_len=[0, 5, max(Nq - 2, 0), Nq + 3, 0],
           prefix=prefix, causal=causal, seed=Nq, **pad(wide))
    if prefix == 0:
        o = P.run(p)
        torch.cuda.synchronize()
        assert int(o[0].count_nonzero()) == 0


def test_everything_empty():
    go(B=2, H=2, Hkv=2, D=128, Nq=3, page=16, q_len=[0, 0], kv_len=[0, 0])
    go(B=2, H=2, Hkv=2, D=128, Nq=3, page=16, q_len=[3, 1], kv_len=[0, 0])


@pytest.mark.parametrize("causal", [True, False])
def test_lengths_left_out_and_out_of_range(causal):
    """None means all; what is out of range is clamped."""
    G.ensure_built()
    page, W, N = 16, 5, 3
    p = P.make(B=2, H=4, Hkv=2, D=64, Nq=N, page=page, kv_len=[W * page] * 2, prefix=2 * page, causal=causal,
               table_pad=0, seed=3)
    ref = P.run(p)
    o = torch.full_like(ref, 7.0)
    cache = S.PageCache(p.cache_k, p.cache_v)
    ws = S.alloc_paged_workspace(2, 4, 2, N, 64)
    S.sage_attn_paged(p.q, o, cache, p.table, ws, prefix_table=p.prefix_table, causal=causal)
    P.check(p, o)
    assert torch.equal(o, ref)
    far = torch.tensor([1 << 30, W * page + 1], dtype=torch.int32, device="cuda")
    o2 = torch.full_like(ref, 7.0)
    S.sage_attn_paged(p.q, o2, cache, p.table, ws, q_len=far, kv_len=far, prefix_table=p.prefix_table,
                      prefix_len=far[:1], causal=causal)
    torch.cuda.synchronize()
    assert torch.equal(o2, ref)
    neg = torch.tensor([-1, -2], dtype=torch.int32, device="cuda")
    o3 = torch.full_like(ref, 7.0)
    S.sage_attn_paged(p.q, o3, cache, p.table, ws, kv_len=neg, prefix_table=p.prefix_table, prefix_len=neg[:1],
                      causal=causal)
    torch.cuda.synchronize()
    assert int(o3.count_nonzero()) == 0


@pytest.mark.parametrize("B,Nq,H,prefix", [(6, 1, 8, 300), (6, 1, 128, 300), (6, 60, 8, 300), (50, 1, 8, 2700), (30, 5, 16, 4200)])
def test_prefix_without_own_table(B, Nq, H, prefix):
    G.ensure_built()
    p = P.make(B=B, H=H, Hkv=4, D=128, Nq=Nq, page=32, kv_len=[0] * B, prefix=prefix, seed=5)
    p.table = None
    P.check(p, P.run(p))


@pytest.mark.parametrize("scale,sm_scale", [(30.0, 0.0), (1.0, 2.0), (0.01, 0.0), (1.0, 1e-6)])
@pytest.mark.parametrize("Nq", [1, 64])
def test_sharp_and_flat_softmax(scale, sm_scale, Nq):
    go(B=2, H=8, Hkv=2, D=128, Nq=Nq, page=16, kv_len=[Nq + 300, Nq + 41], prefix=77, scale=scale, sm_scale=sm_scale,
       seed=11)


@pytest.mark.parametrize("poison", [float("inf"), -float("inf"), 3e38])
def test_other_values_behind_the_lengths(poison):
    go(B=3, H=4, Hkv=2, D=64, Nq=1, page=128, kv_len=[5, 129, 300], prefix=130, poison=poison, seed=12)
    go(B=3, H=4, Hkv=2, D=128, Nq=70, page=128, kv_len=[75, 129, 300], prefix=130, poison=poison, seed=13)


@pytest.mark.parametrize("B,H,Hkv,D,Nq,n,prefix", [
    (1, 4, 2, 128, 1, 40000, 0), (2, 8, 1, 64, 1, 20000, 9000), (40, 8, 2, 128, 1, 1500, 5000),
    (1, 2, 1, 128, 700, 3000, 2000), (3, 6, 2, 64, 300, 900, 0), (16, 8, 2, 128, 4, 300, 3000)])
def test_long_and_many(B, H, Hkv, D, Nq, n, prefix):
    kv = [max(Nq, n - 313 * b % n) for b in range(B)]
    go(B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=64, kv_len=kv, prefix=prefix, seed=n)


@pytest.mark.parametrize("B,Nq,prefix", [(4, 1, 0), (4, 1, 500), (4, 100, 500), (64, 1, 8300), (40, 6, 4300)])
def test_strided_views(B, Nq, prefix):
    """q inside a fused projection, o inside a wider buffer, table rows apart."""
    G.ensure_built()
    H, Hkv, D = 8, 2, 64
    kv = [Nq + (9, 0, 200, 31)[b % 4] for b in range(B)]
    p = P.make(B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=16, kv_len=kv, prefix=prefix, seed=21)
    fused = torch.zeros((B, Nq, H + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    fused[:, :, :H] = p.q.permute(0, 2, 1, 3)
    p.q = fused[:, :, :H].permute(0, 2, 1, 3)
    wide = torch.full((B, p.table.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :p.table.shape[1]] = p.table
    p.table = wide[:, :p.table.shape[1]]
    buf = torch.full((B, H, Nq + 2, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    P.check(p, P.run(p, o=buf[:, :, 1:Nq + 1, :D]))
    assert bool((buf[:, :, 0] == 7).all()) and bool((buf[:, :, -1] == 7).all()) and bool((buf[..., D:] == 7).all())


@pytest.mark.parametrize("B,Nq,H,prefix", [(2, 1, 4, 0), (2, 1, 4, 100), (2, 90, 4, 0), (2, 1, 128, 100), (64, 1, 4, 4200),
                                           (24, 5, 8, 4200)])
def test_a_page_outside_the_cache_reads_as_zeros_and_is_reported(B, Nq, H, prefix):
    G.ensure_built()
    p = P.make(B=B, H=H, Hkv=2, D=128, Nq=Nq, page=16, kv_len=[Nq + 100, Nq + 60] * (B // 2), prefix=prefix, poison=0.0,
               seed=31)
    zero = p.cache_k.shape[0]                              # a page of zeros, added to the definition's cache only
    good = P.Paged(**{**p.__dict__})
    good.cache_k = torch.cat((p.cache_k, torch.zeros_like(p.cache_k[:1])))
    good.cache_v = torch.cat((p.cache_v, torch.zeros_like(p.cache_v[:1])))
    for bad in (zero, -1, 2 ** 31 - 1, -2 ** 31):
        p.table[1, 2] = bad
        good.table = p.table.clone()
        good.table[1, 2] = zero
        if prefix:
            p.prefix_table[3] = bad
            good.prefix_table = p.prefix_table.clone()
            good.prefix_table[3] = zero
        o = P.run(p)
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_ERR_PAGE
        P.check(good, o)


@pytest.mark.parametrize("B,H,Hkv,Nq,n,prefix", [(8, 8, 2, 1, 3000, 0), (40, 8, 2, 1, 500, 3000), (70, 8, 2, 1, 500, 4000), (2, 4, 2, 200, 2000, 700),
                                                  (30, 8, 2, 5, 500, 4000)])
def test_equal_inputs_give_equal_bits(B, H, Hkv, Nq, n, prefix):
    G.ensure_built()
    p = P.make(B=B, H=H, Hkv=Hkv, D=128, Nq=Nq, page=32, kv_len=[Nq + max(0, n - 71 * b) for b in range(B)], prefix=prefix,
               seed=41)
    first = P.run(p).clone()
    ws = S.alloc_paged_workspace(B, H, Hkv, Nq, 128)
    for fill in (0, 0x7F, 0xFF):                           # whatever the workspace held
        ws.fill_(fill)
        assert torch.equal(P.run(p, workspace=ws), first)


@pytest.mark.parametrize("B,Nq,prefix", [(3, 1, 0), (3, 1, 700), (3, 130, 700), (60, 1, 4700), (30, 5, 4700)])
def test_captured_and_replayed_with_growing_lengths(B, Nq, prefix):
    """One graph, captured once, serves every later length: the lengths are read on the device."""
    G.ensure_built()
    H, Hkv, D = 8, 2, 128
    long = [Nq + 400, Nq + 17, Nq + 250] * (B // 3)
    p = P.make(B=B, H=H, Hkv=Hkv, D=D, Nq=Nq, page=16, kv_len=long, prefix=prefix, seed=51)
    cache = S.PageCache(p.cache_k, p.cache_v)
    ws = S.alloc_paged_workspace(B, H, Hkv, Nq, D)
    o = torch.zeros((B, Nq, H, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    q_len = torch.tensor([Nq] * B, dtype=torch.int32, device="cuda")
    kv_len = torch.tensor(long, dtype=torch.int32, device="cuda")
    plen = torch.tensor([prefix], dtype=torch.int32, device="cuda") if prefix else None

    def call():
        S.sage_attn_paged(p.q, o, cache, p.table, ws, q_len=q_len, kv_len=kv_len, prefix_table=p.prefix_table,
                          prefix_len=plen)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]    # two graphs over one workspace, replayed in order
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for k, lens in enumerate(([Nq] * B, [Nq + 400, Nq + 3, Nq + 99] * (B // 3), long)):
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        o.fill_(7.0)
        graphs[k % 2].replay()
        p.kv_len = lens
        P.check(p, o)
        graphs[1 - k % 2].replay()
        P.check(p, o)


def test_two_streams_with_their_own_workspaces():
    G.ensure_built()
    ps = [P.make(B=6, H=8, Hkv=2, D=128, Nq=1, page=16, kv_len=[900 - 100 * b for b in range(6)], prefix=pre, seed=61 + pre)
          for pre in (0, 400)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    wss = [S.alloc_paged_workspace(6, 8, 2, 1, 128) for _ in ps]
    outs = [torch.full((6, 1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3) for _ in ps]
    lens = [torch.tensor(p.kv_len, dtype=torch.int32, device="cuda") for p in ps]
    pl = torch.tensor([400], dtype=torch.int32, device="cuda")
    caches = [S.PageCache(p.cache_k, p.cache_v) for p in ps]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, s, ws, o, n, c in zip(ps, streams, wss, outs, lens, caches):
            S.sage_attn_paged(p.q, o, c, p.table, ws, kv_len=n, prefix_table=p.prefix_table,
                              prefix_len=pl if p.prefix_table is not None else None, stream=s)
    for p, o in zip(ps, outs):
        P.check(p, o)


def test_every_form_at_once():
    """Calls of all forms in flight together, each on its own stream, over and over."""
    G.ensure_built()
    shapes = [dict(B=3, Nq=300, kv=700, prefix=0, pad=2), dict(B=3, Nq=300, kv=700, prefix=130, pad=1200),
              dict(B=4, Nq=40, kv=500, prefix=0, pad=2), dict(B=30, Nq=5, kv=90, prefix=4700, pad=2),
              dict(B=6, Nq=1, kv=900, prefix=0, pad=2), dict(B=6, Nq=1, kv=900, prefix=50, pad=1200),
              dict(B=60, Nq=1, kv=90, prefix=4700, pad=2)]
    H, Hkv, D = 8, 2, 128
    calls = []
    for x in shapes:
        p = P.make(B=x["B"], H=H, Hkv=Hkv, D=D, Nq=x["Nq"], page=16, prefix=x["prefix"], table_pad=x["pad"],
                   kv_len=[x["Nq"] + (x["kv"] - 31 * b) % x["kv"] for b in range(x["B"])], seed=x["kv"])
        want = P.run(p).clone()
        calls.append((p, want, S.alloc_paged_workspace(x["B"], H, Hkv, x["Nq"], D), torch.zeros_like(want),
                      torch.tensor(p.kv_len, dtype=torch.int32, device="cuda"),
                      torch.tensor([x["prefix"]], dtype=torch.int32, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(15):
        for p, _, ws, o, n, pre, s in calls:
            S.sage_attn_paged(p.q, o, S.PageCache(p.cache_k, p.cache_v), p.table, ws, kv_len=n,
                              prefix_table=p.prefix_table, prefix_len=pre if p.prefix_table is not None else None, stream=s)
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    for _, want, _, o, _, _, _ in calls:
        assert torch.equal(o, want)


def test_padding_rows_of_q_and_stale_outputs_do_not_matter():
    """NaN in the query rows behind q_len, and in the output before the call."""
    G.ensure_built()
    for Nq, H in ((3, 4), (50, 4), (200, 2)):
        p = P.make(B=3, H=H, Hkv=2, D=64, Nq=Nq, page=32, q_len=[Nq, 1, Nq // 2], kv_len=[Nq + 70, 40, Nq], prefix=45, seed=Nq)
        for b, n in enumerate(p.q_len):
            p.q[b, :, n:] = float("nan")
        o = torch.full((3, Nq, H, 64), float("nan"), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
        P.run(p, o=o)
        for b, n in enumerate(p.q_len):
            assert bool(o[b, :, n:].isnan().all())
            o[b, :, n:] = 7.0
        P.check(p, o)


def test_waits_for_what_the_stream_waits_for():
    """Lengths, tables, keys and q written just before, by kernels of this stream and by another stream's."""
    G.ensure_built()
    for B, Nq, prefix in ((4, 1, 0), (3, 60, 100), (64, 1, 4300), (30, 5, 4300)):
        p = P.make(B=B, H=8, Hkv=2, D=128, Nq=Nq, page=16, kv_len=[Nq + 300 - 2 * b for b in range(B)], prefix=prefix, seed=B)
        want = P.run(p).clone()
        torch.cuda.synchronize()
        keep = [t.clone() for t in (p.q, p.cache_k, p.cache_v, p.table)]
        other, big = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
        for _ in range(3):
            for t in (p.q, p.cache_k, p.cache_v):
                t.fill_(float("nan"))
            p.table.fill_(0)
            torch.cuda.synchronize()
            with torch.cuda.stream(other):
                for _ in range(4):
                    big = big @ big * 1e-3
                for t, k in zip((p.q, p.cache_k, p.cache_v, p.table), keep):
                    t.copy_(k)
                done = other.record_event()
            torch.cuda.current_stream().wait_event(done)
            assert torch.equal(P.run(p), want)
            p.q.copy_(keep[0] * 0)
            P.run(p)
            p.q.copy_(keep[0])
            assert torch.equal(P.run(p), want)
    assert S.sage_get_device_status() == S.SAGE_OK


def test_a_withheld_copy_times_out_and_the_context_survives():
    """The many-rows kernel's bounded waits, on a few CTAs (about a second each)."""
    G.ensure_built()
    for D, Nq, list_ in ((128, 40, 0), (64, 40, 1), (128, 300, 1), (64, 300, 0)):
        p = P.make(B=1, H=2, Hkv=1, D=D, Nq=Nq, page=64, kv_len=[Nq + 100], seed=D, **pad(list_))
        S.sage_debug_inject_fault(1)
        P.run(p)
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_ERR_TIMEOUT
        P.check(p, P.run(p))


def test_cache_offsets_behind_two_to_the_32_elements():
    G.ensure_built()
    heads, D, page = 32, 128, 128
    pages = 2 ** 32 // (heads * D * page) + 4
    k = torch.zeros((pages, page, heads, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    v = torch.zeros((pages, page, heads, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    g = torch.Generator(device="cuda").manual_seed(5)
    for Nq in (1, 40):
        n = [Nq + 200, Nq + 90]
        last = torch.tensor([[pages - 1, pages - 3, pages - 2], [0, pages - 4, 5]], dtype=torch.int32, device="cuda")
        for pg in last.unique().tolist():
            k[pg] = torch.randn((heads, page, D), device="cuda", generator=g).to(torch.bfloat16)
            v[pg] = torch.randn((heads, page, D), device="cuda", generator=g).to(torch.bfloat16)
        q = torch.randn((2, heads, Nq, D), device="cuda", generator=g).to(torch.bfloat16)
        p = P.Paged(q, k, v, last, [Nq, Nq], n, None, 0, True)
        P.check(p, P.run(p))


def test_convenience_call_and_launch_count():
    G.ensure_built()
    p = P.make(B=2, H=4, Hkv=2, D=64, Nq=2, page=16, kv_len=[50, 3], seed=71)
    kv = torch.tensor(p.kv_len, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = S.attention_paged(p.q, S.PageCache(p.cache_k, p.cache_v), p.table, kv_len=kv, stream=s)
    s.synchronize()
    assert 1 <= S.sage_last_launch_count() <= 3
    P.check(p, o)


@pytest.mark.parametrize("D", [64, 128])
def test_the_widest_tables(D):
    """9 (B * heads) * (tokens / 16 + 6) tiles just below 2^30 are served, one page more is refused."""
    G.ensure_built()
    B, page, W = 3, 128, (((2 ** 30 - 1) // 9 - 6) * 16) // 128
    p = P.make(B=B, H=6, Hkv=3, D=D, Nq=1, page=page, kv_len=[40000, 0, 77], seed=9)
    row = torch.full((1, W + 1), 1 << 30, dtype=torch.int32, device="cuda")
    own = p.table[0, :-(-40000 // page)]
    row[0, :own.numel()] = own
    p.table, p.kv_len = row[:, :W].expand(B, W), [40000, 0, 39999]     # one list of pages for all
    P.check(p, P.run(p))
    p.table = row.expand(B, W + 1)
    with pytest.raises(S.SageError) as e:
        P.run(p)
    assert e.value.code == S.SAGE_ERR_UNSUPPORTED


@pytest.mark.parametrize("Nq,wide_", [(1, 0), (1, 1), (40, 0), (300, 0), (300, 1)])
@pytest.mark.parametrize("top", [2.0 ** 29, -2.0 ** 28])
def test_scores_of_two_to_the_29(Nq, wide_, top):
    """The largest score lies so far above the others that the output is its value: one
    rounding of its weight and one of the output, whatever its distance to the rounded maximum."""
    G.ensure_built()
    D, n, at = 128, 230, 137                               # key `at` has the score `top`, the others half or twice that
    p = P.make(B=1, H=4, Hkv=2, D=D, Nq=Nq, page=16, kv_len=[n], causal=False, sm_scale=1.0, seed=29, **pad(wide_))
    rest = top / 2 if top > 0 else top * 2
    p.q.fill_(2.0 ** 14)
    for j in range(n):
        pg, row = int(p.table[0, j // 16]), j % 16
        p.cache_k[pg, :, row] = (top if j == at else rest) / 2.0 ** 14 / D
    value = p.cache_v[int(p.table[0, at // 16]), :, at % 16].double().repeat_interleave(2, 0)[None, :, None]
    o = P.run(p).double()
    tol = ((1 + P.U_BF16) * (1 + P.U_BF16 + 2.0 ** -18) - 1) * value.abs()
    assert bool(((o - value).abs() <= tol).all())
    assert S.sage_get_device_status() == S.SAGE_OK
