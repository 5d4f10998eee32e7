"""The page-cache operators together, as a serving loop runs them: prompts in
pieces, then single tokens, the pages and slots of every step made on the GPU
from the lengths, and every step's output against plain attention over the
tokens so far."""
import math
import random

import pytest
import torch

import quantized_exact_attention_gb300 as S
from tests import gpu_support as G
from tests import paged_support as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,Hkv,D,page,prefix", [(3, 8, 2, 128, 16, 0), (5, 4, 4, 64, 32, 75), (12, 16, 2, 128, 64, 200)])
def test_serving_loop(B, H, Hkv, D, page, prefix):
    G.ensure_built()
    r = random.Random(B)
    g = torch.Generator(device="cuda").manual_seed(B)
    pieces = [[r.choice((0, 1, 17, 70)) for _ in range(B)] for _ in range(3)] + [[r.choice((0, 1)) for _ in range(B)]
                                                                                 for _ in range(6)]
    longest = sum(max(p) for p in pieces)
    W = -(-longest // page)
    n_pages = B * W + -(-prefix // page) + 5
    cache = S.alloc_page_cache(n_pages, page, Hkv, D)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    ptable, plen, used = None, None, 0
    pk = pv = torch.empty((0, Hkv, D), dtype=torch.bfloat16, device="cuda")
    if prefix:                                             # the shared prompt: one request's tables, kept as the prefix
        t = torch.empty((1, -(-prefix // page)), dtype=torch.int32, device="cuda")
        s = torch.empty((1, prefix), dtype=torch.int32, device="cuda")
        taken = S.sage_page_tables(i32([prefix]), page, order, t, s)
        pk, pv = randn(prefix, Hkv, D), randn(prefix, Hkv, D)
        S.sage_cache_append(pk[None].transpose(1, 2), pv[None].transpose(1, 2), s, cache)
        ptable, plen, used = t[0], i32([prefix]), int(taken)
    table = torch.empty((B, W), dtype=torch.int32, device="cuda")
    have = [0] * B
    ks, vs = ([torch.empty((0, Hkv, D), dtype=torch.bfloat16, device="cuda")] * B for _ in range(2))
    for new in pieces:
        N = max(max(new), 1)
        slots = torch.empty((B, N), dtype=torch.int32, device="cuda")
        old, have = have, [a + n for a, n in zip(have, new)]
        taken = S.sage_page_tables(i32(have), page, order[used:], table, slots, old_len=i32(old))
        q, k, v = randn(B, H, N, D), randn(B, Hkv, N, D), randn(B, Hkv, N, D)
        S.sage_cache_append(k, v, slots, cache)
        o = S.attention_paged(q, cache, table, q_len=i32(new), kv_len=i32(have), prefix_table=ptable, prefix_len=plen)
        torch.cuda.synchronize()
        used += int(taken)
        assert S.sage_get_device_status() == S.SAGE_OK
        ks = [torch.cat((a, k[b, :, :n].transpose(0, 1))) for b, (a, n) in enumerate(zip(ks, new))]
        vs = [torch.cat((a, v[b, :, :n].transpose(0, 1))) for b, (a, n) in enumerate(zip(vs, new))]
        for b, n in enumerate(new):
            assert int(o[b, :, n:].count_nonzero()) == 0
            kk = torch.cat((pk, ks[b])).double().repeat_interleave(H // Hkv, 1).transpose(0, 1)
            vv = torch.cat((pv, vs[b])).double().repeat_interleave(H // Hkv, 1).transpose(0, 1)
            L = kk.shape[1]
            if n == 0:
                continue
            s = q[b, :, :n].double() @ kk.transpose(1, 2) / math.sqrt(D)
            i, j = torch.arange(n, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
            w = torch.softmax(s.masked_fill(j > i + (L - n), -math.inf), -1)
            want, size = w @ vv, w @ vv.abs()
            # output rounding, weight rounding, and 2^-11 for the FP32 scores (|s| stays below 2^4 here)
            tol = P.U_BF16 * want.abs() + (P.U_BF16 * 1.01 + 2.0 ** -11) * size
            assert bool(((o[b, :, :n].double() - want).abs() <= tol).all())
    assert used <= n_pages


def test_a_decode_step_captured_whole():
    """Tables, append and attention in one graph: replayed with the lengths, the
    free list and the tokens of each step, it leaves what the eager calls leave."""
    G.ensure_built()
    B, H, Hkv, D, page, W, steps = 6, 8, 2, 128, 16, 4, 24
    n_pages = B * W
    g = torch.Generator(device="cuda").manual_seed(7)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = [0, 5, 15, 16, 31, 38]

    class Side:
        """One cache with its step's buffers."""
        def __init__(self):
            self.cache = S.alloc_page_cache(n_pages, page, Hkv, D)
            self.cache.k.zero_()
            self.cache.v.zero_()
            self.table = torch.empty((B, W), dtype=torch.int32, device="cuda")
            self.slots = torch.empty((B, 1), dtype=torch.int32, device="cuda")
            self.taken = torch.empty(1, dtype=torch.int32, device="cuda")
            self.q = torch.zeros((B, H, 1, D), dtype=torch.bfloat16, device="cuda")
            self.k = torch.zeros((B, Hkv, 1, D), dtype=torch.bfloat16, device="cuda")
            self.v = torch.zeros_like(self.k)
            self.o = torch.zeros_like(self.q)
            self.old, self.new, self.free = i32([0] * B), i32([0] * B), order.clone()
            self.ws = S.alloc_paged_workspace(B, H, Hkv, 1, D)

        def step(self, stream=None):
            S.sage_page_tables(self.new, page, self.free, self.table, self.slots, self.taken, old_len=self.old,
                               stream=stream)
            S.sage_cache_append(self.k, self.v, self.slots, self.cache, stream=stream)
            S.sage_attn_paged(self.q, self.o, self.cache, self.table, self.ws, kv_len=self.new, stream=stream)

        def begin(self):
            """Pages of the tokens before the first step (whose keys are zero)."""
            S.sage_page_tables(i32(starts), page, order, self.table, None, self.taken)
            torch.cuda.synchronize()
            return int(self.taken)

    eager, whole = Side(), Side()
    whole.step()                                           # the first call, before the capture: no token yet
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        whole.step()
    used = eager.begin()
    assert whole.begin() == used
    have = list(starts)
    for n in range(steps):
        old, have = have, [a + (n + b) % 2 for b, a in enumerate(have)]
        q, k, v = (torch.randn((B, h, 1, D), device="cuda", generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv))
        for x in (eager, whole):
            for dst, src in ((x.q, q), (x.k, k), (x.v, v), (x.old, i32(old)), (x.new, i32(have)),
                             (x.free, torch.cat((order[used:], order[:used])))):
                dst.copy_(src)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_OK
        used += int(eager.taken)
        assert used <= n_pages
        for a, b in ((eager.taken, whole.taken), (eager.table, whole.table), (eager.slots, whole.slots),
                     (eager.o, whole.o), (eager.cache.k, whole.cache.k), (eager.cache.v, whole.cache.v)):
            assert torch.equal(a, b)
    assert int(eager.o.count_nonzero()) > 0


@pytest.mark.parametrize("B,H,Hkv,D,Nq,keys,prefix,pad", [
    (4, 8, 2, 128, 1, 300, 0, 0),                          # clusters
    (4, 8, 2, 128, 1, 300, 60, 1200),                      # few rows from a list
    (40, 16, 8, 128, 1, 60, 1000, 2),                      # ... beside the prefix's list
    (30, 8, 2, 128, 5, 90, 4300, 2),                       # the prefix's items and the requests' in one list
    (3, 4, 2, 64, 40, 500, 0, 2),                          # many rows, whole items
    (3, 4, 2, 128, 300, 700, 130, 1200)])                  # ... from a list
def test_steps_in_flight(B, H, Hkv, D, Nq, keys, prefix, pad):
    """Steps that rebuild the tables from another order of the pages and write
    every key again, one table, slot map, cache and workspace for all of them:
    enqueued without a wait between them, and as one graph replayed at once, they
    leave what they leave one by one."""
    G.ensure_built()
    page, steps = 16, 10
    r, g = random.Random(B), torch.Generator(device="cuda").manual_seed(B)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    N, wp = Nq + keys, -(-prefix // page)
    W = -(-N // page) + pad
    n_pages = wp + B * -(-N // page) + 3
    lens = [[Nq + r.randrange(keys + 1) for _ in range(B)] for _ in range(steps)]
    new = [i32(x) for x in lens]
    order = [torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32) for _ in range(steps)]
    q, k, v = ([randn(B, h, n, D) for _ in range(steps)] for h, n in ((H, Nq), (Hkv, N), (Hkv, N)))
    pk, pv = ([randn(1, Hkv, max(prefix, 1), D) for _ in range(steps)] for _ in range(2))
    plen = i32([prefix])
    cache = S.alloc_page_cache(n_pages, page, Hkv, D)
    ws = S.alloc_paged_workspace(B, H, Hkv, Nq, D)
    table, slots = (torch.empty((B, n), dtype=torch.int32, device="cuda") for n in (W, N))
    ptable, pslots = (torch.empty((1, max(n, 1)), dtype=torch.int32, device="cuda") for n in (wp, prefix))
    taken, ptaken = (torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(2))
    o = [torch.empty((B, Nq, H, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3) for _ in range(steps)]

    def step(n):
        if prefix:
            S.sage_page_tables(plen, page, order[n][:wp], ptable, pslots, ptaken)
            S.sage_cache_append(pk[n], pv[n], pslots, cache)
        S.sage_page_tables(new[n], page, order[n][wp:], table, slots, taken)
        S.sage_cache_append(k[n], v[n], slots, cache)
        S.sage_attn_paged(q[n], o[n], cache, table, ws, kv_len=new[n], prefix_table=ptable[0] if prefix else None,
                          prefix_len=plen if prefix else None)

    def reset():
        for t in (table, slots, ptable, pslots, taken, *o):
            t.fill_(0)
        for t in (cache.k, cache.v):
            t.fill_(float("nan"))
        torch.cuda.synchronize()

    def left():
        torch.cuda.synchronize()
        assert S.sage_get_device_status() == S.SAGE_OK
        return [t.clone().view(torch.int16) for t in (*o, cache.k.contiguous(), cache.v.contiguous())] + [
            t.clone() for t in (table, slots, taken)]

    reset()
    for n in range(steps):
        step(n)
        P.check(P.Paged(q[n], cache.k, cache.v, table, [Nq] * B, lens[n], ptable[0] if prefix else None, prefix, True), o[n])
    want = left()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for n in range(steps):
            step(n)
    for _ in range(3):
        reset()
        for n in range(steps):
            step(n)
        assert all(torch.equal(a, b) for a, b in zip(left(), want))
        reset()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(left(), want))
    for _ in range(4):                                     # replays behind one another
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(left()[:steps], want))
