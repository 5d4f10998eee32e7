"""The operators of drafted trees together, as a serving loop runs them: a
rotated prompt, then steps of tables, tree tables, rotation, append, attention
and the move of the accepted path, each step's output against plain attention
over the tokens that lie on the path to each row."""
import math
import random

import pytest
import torch

import quantized_exact_attention_gb300 as S
from tests import gpu_support as G
from tests import paged_support as P
from tests import tree_support as T

pytestmark = pytest.mark.gpu


class Loop:
    """A batch of requests with its cache; `step` runs one drafted tree of each on the GPU alone."""

    def __init__(self, B, H, Hkv, D, page, N, longest, rotary):
        self.B, self.H, self.Hkv, self.D, self.page, self.N, self.rotary = B, H, Hkv, D, page, N, rotary
        W = -(-longest // page)
        self.cache = S.alloc_page_cache(B * W + 2, page, Hkv, D)
        self.cache.k.fill_(float("nan"))
        self.cache.v.fill_(float("nan"))
        e = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        # every request's pages are its own from the start, so a step only grows into them
        self.free = torch.randperm(B * W, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.table, self.slots, self.taken = e(B, W), e(B, N), e(1)
        self.old, self.new, self.n, self.parents, self.kept = e(B), e(B), e(B), e(B, N), e(B, N)
        self.mask, self.depth = e(B, N, -(-N // 32)), e(B, N)
        z = lambda h: torch.zeros((B, N, h, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)  # noqa: E731
        self.q, self.k, self.v, self.turned, self.o = z(H), z(Hkv), z(Hkv), z(H), z(H)
        self.ws = S.alloc_paged_workspace(B, H, Hkv, N, D)

    def draft(self):
        S.sage_page_tables(self.new, self.page, self.free, self.table, self.slots, self.taken, old_len=self.old)
        S.sage_tree_tables(self.parents, self.mask, self.depth, n_len=self.n)
        S.sage_rope(self.q, self.turned, self.rotary, positions=self.depth, start=self.old, n_len=self.n)
        S.sage_cache_append_rope(self.k, self.v, self.slots, self.cache, self.rotary, positions=self.depth, start=self.old)
        S.sage_attn_paged_tree(self.turned, self.o, self.cache, self.table, self.mask, self.ws, q_len=self.n, kv_len=self.new)

    def accept(self):
        S.sage_cache_keep(self.kept, self.slots, self.cache)


def run(B, H, Hkv, D, page, N, steps, interleaved, captured):
    G.ensure_built()
    r, g = random.Random(B), torch.Generator(device="cuda").manual_seed(B)
    f, a = S.rotary_frequencies(D // 2, scale=4.0, method="parts", trained=64)
    x = Loop(B, H, Hkv, D, page, N, 40 + steps * N, S.make_rotary(f, interleaved=interleaved, amplitude=a))
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    # each request keeps its pages: its part of the free list is where its table takes them from
    W = x.table.shape[1]
    x.table.copy_(x.free.reshape(B, W))
    own = x.table.clone()
    have = [0] * B
    ks, vs = ([torch.empty((0, Hkv, D), dtype=torch.float64, device="cuda")] * B for _ in range(2))
    graphs = None
    for step in range(steps):
        n = [r.choice((N, N, 1, r.randint(1, N))) for _ in range(B)]
        parents = [T.random_parents(r, N, r.choice((0, 2, 5))) for _ in range(B)]
        sees = [T.sees_of(p) for p in parents]
        # the accepted path: from a root of the tree down to some token
        paths = [sorted(sees[b][r.randrange(n[b])]) for b in range(B)]
        x.old.copy_(T.i32(have))
        x.new.copy_(T.i32([h + m for h, m in zip(have, n)]))
        x.n.copy_(T.i32(n))
        x.parents.copy_(T.i32(parents))
        x.kept.copy_(T.i32([p + [-1] * (N - len(p)) for p in paths]))
        for t in (x.q, x.k, x.v):
            t.copy_(randn(*t.shape))
        # tables of the step from pages the requests own: what old_len covers is kept, the rest taken in order
        need = [-(-(h + m) // page) - -(-h // page) for h, m in zip(have, n)]
        take = [int(p) for b in range(B) for p in own[b, -(-have[b] // page):-(-have[b] // page) + need[b]]]
        x.free[:len(take)] = T.i32(take) if take else x.free[:0]
        x.o.fill_(7.0)
        last = x.turned.clone()
        if captured and step == 1:
            torch.cuda.synchronize()
            graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
            with torch.cuda.graph(graphs[0]):
                x.draft()
            with torch.cuda.graph(graphs[1]):
                x.accept()
        if graphs:
            graphs[0].replay()
        else:
            x.draft()
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_OK
        assert int(x.taken) == sum(need)
        pos = [[have[b] + len(sees[b][i]) - 1 for i in range(N)] for b in range(B)]
        angle = T.angles(pos, f)
        tq, q_off = T.turned(x.q, angle, D // 2, interleaved, a)
        tk, k_off = T.turned(x.k, angle, D // 2, interleaved, a)
        slots = x.slots.long()
        for b in range(B):
            assert bool((x.o[b, :, n[b]:] == 7.0).all()) and bool((x.turned[b, :, n[b]:] == last[b, :, n[b]:]).all())
            T.near(x.turned[b, :, :n[b]], tq[b, :, :n[b]], q_off[b, :, :n[b]])
            kb, vb = (t[slots[b, :n[b]] // page, :, slots[b, :n[b]] % page] for t in (x.cache.k, x.cache.v))
            T.near(kb.transpose(0, 1), tk[b, :, :n[b]], k_off[b, :, :n[b]])
            assert torch.equal(vb.transpose(0, 1), x.v[b, :, :n[b]])
            kb, vb = kb.double(), vb.double()
            kk, vv = (torch.cat((old, new)).repeat_interleave(H // Hkv, 1).transpose(0, 1)
                      for old, new in ((ks[b], kb), (vs[b], vb)))
            s = x.turned[b, :, :n[b]].double() @ kk.transpose(1, 2) / math.sqrt(D)
            hidden = torch.zeros((n[b], have[b] + n[b]), dtype=torch.bool)
            for i in range(n[b]):
                for t in range(n[b]):
                    hidden[i, have[b] + t] = t not in sees[b][i]
            w = torch.softmax(s.masked_fill(hidden.cuda(), -math.inf), -1)
            want, size = w @ vv, w @ vv.abs()
            # output rounding, weight rounding, and 2^-11 for the FP32 scores (|s| stays below 2^4 here)
            tol = P.U_BF16 * want.abs() + (P.U_BF16 * 1.01 + 2.0 ** -11) * size
            assert bool(((x.o[b, :, :n[b]].double() - want).abs() <= tol).all())
            ks[b], vs[b] = (torch.cat((old, new[paths[b]])) for old, new in ((ks[b], kb), (vs[b], vb)))
        if graphs:
            graphs[1].replay()
        else:
            x.accept()
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_OK
        have = [h + len(p) for h, p in zip(have, paths)]
        for b in range(B):                                 # what the cache holds of the committed tokens
            pages = x.table[b, :-(-have[b] // page)].long()
            k = x.cache.k[pages].permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:have[b]].double()
            v = x.cache.v[pages].permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:have[b]].double()
            assert torch.equal(v, vs[b])
            assert torch.equal(k, ks[b])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,H,Hkv,D,page,N,interleaved", [(3, 8, 2, 128, 16, 12, False), (5, 4, 4, 64, 32, 7, True),
                                                          (2, 16, 2, 128, 64, 40, True)])
def test_drafting_loop(B, H, Hkv, D, page, N, interleaved, captured):
    run(B, H, Hkv, D, page, N, 6, interleaved, captured)


def test_calls_that_allocate_their_outputs():
    """rope, tree_tables and attention_paged with a mask, on the current stream and on one of their own; one launch each."""
    G.ensure_built()
    B, H, Hkv, D, page, N, base = 3, 8, 2, 128, 16, 20, 150
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    rotary = S.make_rotary(S.rotary_frequencies(D)[0])
    r = random.Random(3)
    parents = T.i32([T.random_parents(r, N, 3) for _ in range(B)])
    n = [N, 0, 7]
    cache = S.alloc_page_cache(B * 11, page, Hkv, D)
    cache.k.copy_(randn(*cache.k.shape))
    cache.v.copy_(randn(*cache.v.shape))
    table = torch.randperm(B * 11, generator=torch.Generator().manual_seed(1)).to(torch.int32).reshape(B, 11).cuda()
    q, kv = randn(B, H, N, D), T.i32([base + x for x in n])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for stream in (None, side):
        mask, depth = S.tree_tables(parents, n_len=T.i32(n), stream=stream)
        assert S.sage_last_launch_count() == 1
        torch.cuda.synchronize()
        turned = S.rope(q, rotary, positions=depth, start=T.i32([base] * B), n_len=T.i32(n), stream=stream)
        assert S.sage_last_launch_count() == 1
        torch.cuda.synchronize()
        o = S.attention_paged(turned, cache, table, q_len=T.i32(n), kv_len=kv, mask=mask, stream=stream)
        torch.cuda.synchronize()
        outs.append((mask, depth, turned, o))
        for b in range(B):
            assert int(turned[b, :, n[b]:].count_nonzero()) == 0 and int(o[b, :, n[b]:].count_nonzero()) == 0
            assert int(mask[b, n[b]:].count_nonzero()) == 0
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    mask, _, turned, o = outs[0]
    p = P.Paged(turned, cache.k, cache.v, table, n, [base + x for x in n], None, 0, False)
    T.check(p, [T.sees_of(row) for row in parents.tolist()], o, fill=0.0)


def test_appends_and_moves_on_their_own_streams():
    """Steps of four requests' caches in flight together, each on its own stream, then all as one captured graph."""
    G.ensure_built()
    B, Hkv, D, page, N, K, count = 5, 4, 64, 32, 30, 9, 4
    rotary = S.make_rotary(S.rotary_frequencies(32)[0], interleaved=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    r = random.Random(4)
    first = [[randn(B * 2, page, Hkv, D).permute(0, 2, 1, 3) for _ in range(2)] for _ in range(count)]
    caches = [S.PageCache(*(t.clone() for t in pair)) for pair in first]
    slots = [torch.randperm(B * 2 * page, generator=torch.Generator().manual_seed(i))[:B * N].to(torch.int32).reshape(B, N).cuda()
             for i in range(count)]
    kept = [T.i32([sorted(r.sample(range(N), K)) for _ in range(B)]) for _ in range(count)]
    new = [[randn(B, Hkv, N, D) for _ in range(2)] for _ in range(count)]

    def step(i, stream=None):
        S.sage_cache_append_rope(*new[i], slots[i], caches[i], rotary, stream=stream)
        S.sage_cache_keep(kept[i], slots[i], caches[i], stream=stream)

    def reset():
        for c, pair in zip(caches, first):
            c.k.copy_(pair[0])
            c.v.copy_(pair[1])
        torch.cuda.synchronize()

    def left():
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_OK
        return [t.clone() for c in caches for t in (c.k, c.v)]

    reset()
    for i in range(count):
        step(i)
        torch.cuda.synchronize()
    want = left()
    streams = [torch.cuda.Stream() for _ in range(count)]
    for _ in range(3):
        reset()
        for i in range(count):
            step(i, streams[i])
        assert all(torch.equal(a, b) for a, b in zip(left(), want))
    graph = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(graph):
        for i in range(count):
            step(i)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(left(), want))


def test_a_plan_that_is_not_aligned_is_refused():
    G.ensure_built()
    whole = S.make_rotary(S.rotary_frequencies(64)[0])
    odd = S.Rotary(whole.turns[1:17])                      # 16 pairs that begin 8 bytes behind an aligned address
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(S.SageError) as e:
        S.sage_rope(x, x, odd)
    assert e.value.code == S.SAGE_ERR_UNSUPPORTED
    with pytest.raises(S.SageError):
        S.sage_rope(x, x, S.make_rotary(S.rotary_frequencies(40)[0]))
