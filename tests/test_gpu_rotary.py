"""Rotary positions and the append that rotates, against their definition in 64 bits."""
import math
import random

import pytest
import torch

import quantized_exact_attention_gb300 as S
from tests import gpu_support as G
from tests import tree_support as T

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)


def view(B, H, N, D, layout, seed=0):
    """A [B, H, N, D] view in one of the memory orders."""
    if layout == "nhd":
        return randn(B, N, H, D, seed=seed).permute(0, 2, 1, 3)
    if layout == "hnd":
        return randn(B, H, N, D, seed=seed)
    return randn(B, N, H, 3, D, seed=seed)[:, :, :, 1].permute(0, 2, 1, 3)     # one third of a fused projection


def blank(B, H, N, D, fill=7.0):
    return torch.full((B, N, H, D), fill, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)


def check_rope(x, out, r, f, positions, n_len=None, inverse=False, fill=7.0):
    torch.cuda.synchronize()
    B, H, N, D = x.shape
    want, off = T.turned(x, T.angles(positions, f), 2 * len(f), r.interleaved, r.amplitude, inverse)
    for b in range(B):
        n = N if n_len is None else min(max(n_len[b], 0), N)
        T.near(out[b, :, :n], want[b, :, :n], off[b, :, :n])
        assert torch.equal(out[b, :, :n, 2 * len(f):], x[b, :, :n, 2 * len(f):])
        assert bool((out[b, :, n:] == fill).all()), "rows behind n_len were written"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("D,rd", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 16), (128, 112)])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "fused"])
def test_parts_and_layouts(D, rd, interleaved, inverse, layout):
    G.ensure_built()
    B, H, N = 2, 5, 37
    f = S.rotary_frequencies(rd)[0]
    r = S.make_rotary(f, interleaved=interleaved, amplitude=1.25)
    x, out = view(B, H, N, D, layout), blank(B, H, N, D)
    S.sage_rope(x, out, r, inverse=inverse)
    check_rope(x, out, r, f, [range(N)] * B, inverse=inverse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (3, 1, 33), (1, 2, 7), (5, 3, 1), (2, 8, 19), (1, 24, 65), (2, 33, 3), (64, 32, 1),
                                   (1, 9, 700), (130, 1, 17)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_and_tokens(B, H, N, D, interleaved):
    G.ensure_built()
    f = S.rotary_frequencies(D, 500000.0)[0]
    r = S.make_rotary(f, interleaved=interleaved)
    x, out = view(B, H, N, D, "nhd", seed=H), blank(B, H, N, D)
    start = [(977 * b) % 5000 for b in range(B)]
    S.sage_rope(x, out, r, start=T.i32(start))
    check_rope(x, out, r, f, [range(s, s + N) for s in start])


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions(interleaved):
    """Given for each token, for all requests, strided, negative, far, with and without a start, rows behind n_len."""
    G.ensure_built()
    B, H, N, D = 4, 3, 21, 64
    f = S.rotary_frequencies(D)[0]
    r = S.make_rotary(f, interleaved=interleaved)
    x = view(B, H, N, D, "nhd")
    rnd = random.Random(1)
    far = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7, -1, 0, 1, 10 ** 6 + 3, 123456789]
    pos = [[rnd.choice(far + [rnd.randrange(1 << 20)]) for _ in range(N)] for _ in range(B)]
    start, n_len = [0, 100000, -5, 2 ** 31 - 1], [N, 0, N - 4, N + 9]
    for at, shared in ((T.i32(pos), False), (T.i32(pos[1]), True),
                       (torch.cat((T.i32(pos), T.i32(pos)), 1)[:, :N], False), (T.i32(pos[2])[None].expand(B, N), None)):
        rows = pos if shared is False else [pos[1 if shared else 2]] * B
        out = blank(B, H, N, D)
        S.sage_rope(x, out, r, positions=at)
        check_rope(x, out, r, f, rows)
        out = blank(B, H, N, D)
        S.sage_rope(x, out, r, positions=at, start=T.i32(start), n_len=T.i32(n_len))
        check_rope(x, out, r, f, [[s + p for p in row] for s, row in zip(start, rows)], n_len)
    out = S.rope(x, r, n_len=T.i32([-3, 1, 2, N]))
    check_rope(x, out, r, f, [range(N)] * B, [-3, 1, 2, N], fill=0.0)


@pytest.mark.parametrize("rd", [32, 64])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_in_place(rd, layout):
    G.ensure_built()
    f = S.rotary_frequencies(rd)[0]
    for interleaved in (False, True):
        r = S.make_rotary(f, interleaved=interleaved)
        x = view(3, 6, 50, 64, layout)
        apart = blank(3, 6, 50, 64)
        S.sage_rope(x, apart, r)
        S.sage_rope(x, x, r)
        torch.cuda.synchronize()
        assert torch.equal(x, apart)


def test_forms_of_one_call_agree_bit_for_bit():
    """The split of heads among warps and the place of a token in its warp change nothing."""
    G.ensure_built()
    f = S.rotary_frequencies(128)[0]
    r = S.make_rotary(f, interleaved=False)
    x = view(2, 40, 300, 128, "nhd")
    whole = S.rope(x, r)
    for h in (1, 3, 40):
        for n in (1, 7, 300):
            part = S.rope(x[:, :h, :n], r)
            assert torch.equal(part, whole[:, :h, :n])


@pytest.mark.parametrize("amplitude", [1.0, 2.0 ** -20, 2.0 ** 10])
def test_sines_and_cosines(amplitude):
    """Pairs (1, 0) give the cosine and the sine themselves, at every eighth of a turn and beside it too."""
    G.ensure_built()
    N = 4096
    f = [2 * math.pi / n for n in (3, 5, 8, 16, 64, 100, 1000, 1024)] + [1.0, 0.5, 1e-3, 0.25, 3.0, 7e-5, 0.1, 0.01]
    for interleaved in (False, True):
        r = S.make_rotary(f, interleaved=interleaved, amplitude=amplitude)
        x = torch.zeros((1, 1, N, 64), dtype=torch.bfloat16, device="cuda")
        x[..., slice(0, 32, 2) if interleaved else slice(0, 16)] = 1.0
        check_rope(x, S.rope(x, r), r, f, [range(N)])


def test_special_values_stay_in_their_pair():
    G.ensure_built()
    f = S.rotary_frequencies(32)[0]
    for interleaved in (False, True):
        r = S.make_rotary(f, interleaved=interleaved)
        x = view(1, 2, 4, 64, "nhd")
        first, second = (6, 7) if interleaved else (3, 19)
        x[0, 0, 1, first] = float("nan")
        x[0, 1, 2, second] = float("inf")
        x[0, 0, 3, 40] = float("nan")                       # behind the rotated channels
        x[0, 1, 3, 41] = float("-inf")
        clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
        y, z = S.rope(x, r), S.rope(clean, r)
        touched = torch.zeros_like(x, dtype=torch.bool)
        for h, n in ((0, 1), (1, 2)):
            touched[0, h, n, first] = touched[0, h, n, second] = True
        touched[0, 0, 3, 40] = touched[0, 1, 3, 41] = True
        assert torch.equal(y[~touched], z[~touched])
        assert not bool(torch.isfinite(y[touched]).any())
        assert torch.equal(y[..., 32:].contiguous().view(torch.int16), x[..., 32:].contiguous().view(torch.int16))


def test_gradient():
    """The inverse is the gradient's map: against the formula's gradient, and against differences of the forward map."""
    G.ensure_built()
    B, H, N, D, rd = 2, 4, 30, 64, 48
    f, a = S.rotary_frequencies(rd, scale=8.0, method="parts")
    for interleaved in (False, True):
        r = S.make_rotary(f, interleaved=interleaved, amplitude=a)
        x, g = view(B, H, N, D, "nhd", seed=1), view(B, H, N, D, "hnd", seed=2)
        pos = [range(1000, 1000 + N)] * B
        dx = S.rope(g, r, start=T.i32([1000] * B), inverse=True)
        angle = T.angles(pos, f)
        leaf = x.double().requires_grad_()
        R, half = rd, rd // 2
        c, s = a * torch.cos(angle)[:, None], a * torch.sin(angle)[:, None]
        p, q = (leaf[..., 0:R:2], leaf[..., 1:R:2]) if interleaved else (leaf[..., :half], leaf[..., half:R])
        pair = (p * c - q * s, p * s + q * c)
        y = torch.cat((torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1), leaf[..., R:]), -1)
        y.backward(g.double())
        _, off = T.turned(g, angle, rd, interleaved, a, True)
        T.near(dx, leaf.grad, off)
        # <g, rope(x + e) - rope(x - e)> / 2 = <dx, e>, for steps e = one channel of one row that BF16 holds: each side is
        # off by its roundings, of outputs below 2 * 8 in size here
        for b, h, n, ch in ((0, 0, 0, 0), (1, 3, 29, 47), (0, 2, 11, 24), (1, 1, 5, 63)):
            e = torch.zeros_like(x)
            e[b, h, n, ch] = 4.0
            base = torch.zeros_like(x)
            up, down = S.rope(base + e, r, start=T.i32([1000] * B)), S.rope(base - e, r, start=T.i32([1000] * B))
            assert torch.equal(up, -down)                   # the map is odd, so the differences are exact
            slope = (g.double() * (up.double() - down.double())).sum() / 8.0
            # two outputs of size up to 4 A, each rounded to BF16, times g; dx rounded itself
            tol = 2.0 ** -8 * a * 2 * float(g[b, h, n].abs().max()) + float(dx[b, h, n, ch].abs()) * 2.0 ** -8 + 1e-4
            assert abs(float(slope) - float(dx[b, h, n, ch])) <= tol
        back = S.rope(S.rope(x, r, start=T.i32([1000] * B)), r, start=T.i32([1000] * B), inverse=True)
        want = x.double().clone()
        want[..., :rd] *= a * a
        size = T.turned(x, angle, rd, interleaved, a)[1] * 2.0 ** 21          # A (|x1| + |x2|)
        tol = (a * size + want.abs()) * (2.0 ** -8 * 1.02 + 2.0 ** -19)
        assert bool(((back.double() - want).abs() <= tol).all())


def test_far_strides():
    """Rows over 2^31 elements apart, in the input and in the output."""
    G.ensure_built()
    apart = (1 << 31) + 1024
    buf = torch.empty(apart + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (2, 2, 5, 128), (apart, 128, 256, 1))
    src = randn(2, 2, 5, 128, seed=3)
    x.copy_(src)
    f = S.rotary_frequencies(128)[0]
    r = S.make_rotary(f)
    want = S.rope(src, r)
    assert torch.equal(S.rope(x, r), want)
    S.sage_rope(src, x, r)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,N,D,page,rd", [(1, 1, 1, 64, 16, 64), (64, 8, 1, 128, 16, 128), (5, 2, 40, 128, 32, 64),
                                             (3, 16, 33, 64, 64, 16), (2, 3, 130, 128, 128, 96), (1, 24, 300, 128, 64, 128)])
def test_append(B, H, N, D, page, rd, interleaved, layout):
    """Keys land as sage_rope leaves them, values as they are; every other row of the cache stays."""
    G.ensure_built()
    f = S.rotary_frequencies(rd)[0]
    r = S.make_rotary(f, interleaved=interleaved, amplitude=0.75)
    n_pages = B * -(-N // page) + 3
    shape = (n_pages, page, H, D) if layout == "nhd" else (n_pages, H, page, D)
    ck, cv = randn(*shape, seed=1), randn(*shape, seed=2)
    cache = S.PageCache(*(t.permute(0, 2, 1, 3) if layout == "nhd" else t for t in (ck, cv)))
    kv = randn(B, N, 2, H, D, seed=3)
    k, v = kv[:, :, 0].permute(0, 2, 1, 3), kv[:, :, 1].permute(0, 2, 1, 3)
    slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(N))[:B * N].to(torch.int32).reshape(B, N)
    slots[:, N // 2::5] = -1                               # tokens without a place
    if N > 1:
        slots[0, 0] = 5
        slots[slots == 5] = 5
    pos = torch.randint(0, 1 << 20, (B, N), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(N))
    start = T.i32([3 * b for b in range(B)])
    want_k, want_v = cache.k.clone(), cache.v.clone()
    rot = S.rope(k, r, positions=pos, start=start)
    for b in range(B):
        for i in range(N):
            s = int(slots[b, i])
            if s >= 0 and not (s == 5 and (b, i) != (0, 0)):
                want_k[s // page, :, s % page], want_v[s // page, :, s % page] = rot[b, :, i], v[b, :, i]
    slots[(slots == 5).logical_and(torch.arange(B * N).reshape(B, N) > 0)] = -1
    S.sage_cache_append_rope(k, v, slots.cuda(), cache, r, positions=pos, start=start)
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)


def test_append_outside_the_cache_is_recorded():
    G.ensure_built()
    r = S.make_rotary(S.rotary_frequencies(64)[0])
    cache = S.alloc_page_cache(4, 16, 2, 64)
    cache.k.fill_(3.0)
    cache.v.fill_(3.0)
    k = randn(1, 2, 3, 64)
    S.sage_cache_append_rope(k, k, T.i32([[7, 64, 2 ** 31 - 1]]), cache, r)
    assert S.sage_get_device_status() == S.SAGE_ERR_PAGE
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(cache.v[0, :, 7], k[0, :, 0])
    assert torch.equal(cache.k[0, :, 7], S.rope(k, r)[0, :, 0])
    rest = torch.ones((4, 16), dtype=torch.bool, device="cuda")
    rest[0, 7] = False
    for t in (cache.k, cache.v):
        assert bool((t.permute(0, 2, 1, 3)[rest] == 3.0).all())


def test_other_streams_and_graphs():
    """Calls on streams of their own, and one graph replayed with other positions."""
    G.ensure_built()
    B, H, N, D = 3, 8, 50, 128
    r = S.make_rotary(S.rotary_frequencies(D)[0])
    xs = [view(B, H, N, D, "nhd", seed=s) for s in range(4)]
    starts = [T.i32([s * 100 + b for b in range(B)]) for s in range(4)]
    want = [S.rope(x, r, start=s) for x, s in zip(xs, starts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [blank(B, H, N, D) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s, o, st in zip(xs, starts, outs, streams):
            S.sage_rope(x, o, r, start=s, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    x, start, out = xs[0].clone(), starts[0].clone(), blank(B, H, N, D)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.sage_rope(x, out, r, start=start)
    for k in (2, 1, 3):
        x.copy_(xs[k])
        start.copy_(starts[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])


# Few heads and so many tokens that a lane holds rows of 2 or 4 tokens at a time: of 4 tokens from 14,589 tokens on where
# heads fill a warp's lanes (4 of 128 channels, 8 of 64), later where they are fewer; of 2 from 7,295 on, up to twice as
# many heads.  The same rows in calls of a thousand tokens take the form with one.
def whole_and_parts(B, N):
    """Request and token ranges of calls small enough for the form with a token at a time."""
    if N >= 1000:
        return [(slice(b, b + 1), slice(i, i + 1000)) for b in range(B) for i in range(0, N, 1000)]
    many = max(1, 1000 // N)
    return [(slice(b, b + many), slice(0, N)) for b in range(0, B, many)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,N,D,rd,together", [
    (7, 1, 16801, 128, 128, 4), (1, 1, 65536, 128, 64, 4), (3, 3, 5333, 128, 48, 4), (40, 2, 777, 128, 128, 4), (15001, 4, 1, 128, 128, 4),
    (5, 1, 7001, 128, 16, 2), (9, 4, 1001, 128, 112, 2), (1, 8, 8003, 128, 128, 2), (2, 7, 5001, 128, 64, 2),
    (3, 1, 41001, 64, 64, 4), (1, 8, 15001, 64, 16, 4), (4, 5, 3777, 64, 64, 4), (5001, 6, 3, 64, 48, 4),
    (1, 7, 8001, 64, 64, 2), (3, 16, 2500, 64, 32, 2), (2500, 11, 3, 64, 64, 2)])
def test_several_tokens_of_a_lane(B, H, N, D, rd, together, interleaved):
    """Tokens of different requests in one lane, a count that its tokens do not divide, rows behind n_len, in place: the bits
    of the form with one token, and the definition."""
    G.ensure_built()
    apart = 32 // (D // 16) // min(32 // (D // 16), 1 << (H - 1).bit_length())       # tokens beside each other in a warp
    assert -(-B * N // (apart * together)) >= 24 * torch.cuda.get_device_properties(0).multi_processor_count
    r_ = random.Random(B + N)
    f = S.rotary_frequencies(rd, 500000.0)[0]
    r = S.make_rotary(f, interleaved=interleaved, amplitude=1.25)
    x = view(B, H, N, D, "nhd", seed=H)
    gen = torch.Generator(device="cuda").manual_seed(N)
    pos = torch.randint(-(1 << 30), 1 << 30, (B, N), dtype=torch.int32, device="cuda", generator=gen)
    start = torch.randint(0, 1 << 20, (B,), dtype=torch.int32, device="cuda", generator=gen)
    lens = [r_.choice((N, N, N - 1, 0, -1, N + 3, r_.randrange(N + 1))) for _ in range(B)]
    n_len = T.i32(lens)
    live = torch.arange(N, device="cuda")[None] < n_len[:, None]                      # [B, N]
    for inverse in (False, True):
        for at, first in ((None, None), (pos, start)):
            out, parts = blank(B, H, N, D), blank(B, H, N, D)
            S.sage_rope(x, out, r, positions=at, start=first, n_len=n_len, inverse=inverse)
            for bs, ns in whole_and_parts(B, N):
                n = len(range(*ns.indices(N)))
                off = torch.arange(ns.start, ns.start + n, dtype=torch.int32, device="cuda")
                S.sage_rope(x[bs, :, ns], parts[bs, :, ns], r, positions=off if at is None else at[bs, ns],
                            start=None if first is None else first[bs], n_len=n_len[bs] - ns.start, inverse=inverse)
            torch.cuda.synchronize()
            assert torch.equal(out, parts)
            assert bool((out.permute(0, 2, 1, 3)[~live] == 7.0).all()), "rows behind n_len were written"
            there = x.clone(memory_format=torch.preserve_format)
            S.sage_rope(there, there, r, positions=at, start=first, n_len=n_len, inverse=inverse)
            want = torch.where(live[:, None, :, None], out, x)
            assert torch.equal(there, want)
    # and some rows from their definition: the first, the last, those about a border of requests
    for b, i in {(0, 0), (B - 1, max(0, N - 20)), (B // 2, 0), (B // 2, N // 2)}:
        S.sage_rope(x, out, r, positions=pos, start=start)
        some = slice(i, min(N, i + 20))
        p = [[int(start[b]) + int(v) for v in pos[b, some].tolist()]]
        check_rope(x[b:b + 1, :, some], out[b:b + 1, :, some], r, f, p)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,N,D,page,rd", [(9, 4, 1001, 128, 16, 128), (3, 1, 11003, 128, 64, 64), (8001, 3, 1, 128, 32, 128),
                                             (2, 8, 4001, 64, 128, 64), (2501, 5, 3, 64, 16, 16), (20, 2, 777, 128, 16, 48)])
def test_append_several_tokens_of_a_lane(B, H, N, D, page, rd, interleaved):
    """Tokens without a place or with one outside the cache beside tokens that have one, in one lane."""
    G.ensure_built()
    f = S.rotary_frequencies(rd)[0]
    r = S.make_rotary(f, interleaved=interleaved)
    n_pages = -(-B * N // page) + 2
    c0 = S.PageCache(*(randn(n_pages, page, H, D, seed=s).permute(0, 2, 1, 3) for s in (1, 2)))
    c1 = S.PageCache(c0.k.clone(memory_format=torch.preserve_format), c0.v.clone(memory_format=torch.preserve_format))
    kv = randn(B, N, 2, H, D, seed=3)
    k, v = kv[:, :, 0].permute(0, 2, 1, 3), kv[:, :, 1].permute(0, 2, 1, 3)
    cpu = torch.Generator().manual_seed(N)
    slots = torch.randperm(n_pages * page, generator=cpu)[:B * N].to(torch.int32).reshape(B, N)
    kind = torch.randint(0, 6, (B, N), generator=cpu)
    slots[kind == 0] = -1
    slots[kind == 1] = n_pages * page                                                # the first behind the cache
    slots[0, 0] = 2 ** 31 - 1
    gen = torch.Generator(device="cuda").manual_seed(N)
    pos = torch.randint(0, 1 << 20, (B, N), dtype=torch.int32, device="cuda", generator=gen)
    start = torch.randint(0, 1 << 20, (B,), dtype=torch.int32, device="cuda", generator=gen)
    there = slots.cuda()
    S.sage_cache_append_rope(k, v, there, c0, r, positions=pos, start=start)
    assert S.sage_get_device_status() == S.SAGE_ERR_PAGE
    for bs, ns in whole_and_parts(B, N):
        S.sage_cache_append_rope(k[bs, :, ns], v[bs, :, ns], there[bs, ns], c1, r, positions=pos[bs, ns], start=start[bs])
    assert S.sage_get_device_status() == S.SAGE_ERR_PAGE
    assert S.sage_get_device_status() == S.SAGE_OK
    assert torch.equal(c0.k, c1.k) and torch.equal(c0.v, c1.v)
    # and against the rotation of the same rows; all other rows of the cache as they were
    want_k, want_v = (randn(n_pages, page, H, D, seed=s).reshape(-1, H, D) for s in (1, 2))
    held = (there >= 0) & (there < n_pages * page)
    rot = S.rope(k, r, positions=pos, start=start)
    want_k[there[held].long()] = rot.permute(0, 2, 1, 3)[held]
    want_v[there[held].long()] = v.permute(0, 2, 1, 3)[held]
    assert torch.equal(c0.k.permute(0, 2, 1, 3).reshape(-1, H, D), want_k)
    assert torch.equal(c0.v.permute(0, 2, 1, 3).reshape(-1, H, D), want_v)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_the_result_carries_the_gradient(interleaved, inverse):
    """rope of an x that requires a gradient: the bits of a call without, and backward is the inverse form."""
    G.ensure_built()
    B, H, N, D, rd = 3, 4, 29, 64, 48
    f, a = S.rotary_frequencies(rd, scale=8.0, method="parts")
    r = S.make_rotary(f, interleaved=interleaved, amplitude=a)
    x, g = view(B, H, N, D, "fused", seed=1), view(B, H, N, D, "hnd", seed=2)
    start, lens = T.i32([1000, 5, 70000]), [N, 0, N - 3]
    for n_len in (None, T.i32(lens)):
        plain = S.rope(x, r, start=start, n_len=n_len, inverse=inverse)
        assert not plain.requires_grad
        leaf = x.clone().requires_grad_()
        y = S.rope(leaf, r, start=start, n_len=n_len, inverse=inverse)
        assert torch.equal(y, plain)
        y.backward(g)
        want = S.rope(g, r, start=start, n_len=n_len, inverse=not inverse)
        assert torch.equal(leaf.grad, want)
        pos = [range(s, s + N) for s in (1000, 5, 70000)]
        check_rope(g, leaf.grad, r, f, pos, None if n_len is None else lens, not inverse, fill=0.0)
        with torch.no_grad():
            assert not S.rope(leaf, r, start=start, n_len=n_len).requires_grad
    # into another tensor, and further on: the gradient of an expression of it
    leaf = x.clone().requires_grad_()
    (S.rope(leaf, r, start=start, inverse=inverse) * g).float().pow(2).sum().backward()
    y = S.rope(x, r, start=start, inverse=inverse)
    want = S.rope((2 * (y * g).float()).to(torch.bfloat16) * g, r, start=start, inverse=not inverse)
    assert torch.equal(leaf.grad, want)


def test_gradients_of_other_forms():
    """A gradient that is one value expanded, one of other strides, of a gradient, on a stream, in a graph; and differences."""
    G.ensure_built()
    B, H, N, D = 2, 3, 17, 128
    f = S.rotary_frequencies(D)[0]
    r = S.make_rotary(f)
    x = view(B, H, N, D, "nhd", seed=4)
    ones = torch.ones_like(x)
    want = S.rope(ones, r, inverse=True)
    leaf = x.clone().requires_grad_()
    S.rope(leaf, r).sum().backward()
    assert torch.equal(leaf.grad, want)
    g = randn(B, H, D, N, seed=5).transpose(2, 3)          # channels apart
    odd = randn(B * H * N * D + 1, seed=6)[1:].view(B, H, N, D)                       # not on 16 bytes
    for grad in (g, odd, randn(H, N, D, seed=7).expand(B, H, N, D)):
        leaf = x.clone().requires_grad_()
        S.rope(leaf, r).backward(grad)
        assert torch.equal(leaf.grad, S.rope(grad.clone(memory_format=torch.contiguous_format), r, inverse=True))
    # of a gradient: the map is linear, so the gradient's gradient is the map again
    leaf, v = x.clone().requires_grad_(), view(B, H, N, D, "nhd", seed=8).requires_grad_()
    (dx,) = torch.autograd.grad(S.rope(leaf, r), leaf, v, create_graph=True)
    u = view(B, H, N, D, "nhd", seed=9)
    (dv,) = torch.autograd.grad(dx, v, u)
    assert torch.equal(dv, S.rope(u, r))
    # differences of one channel by a step that BF16 holds, from 0: both sides within their roundings
    leaf = torch.zeros_like(x).requires_grad_()
    S.rope(leaf, r).backward(u)
    for b, h, n, c in ((0, 0, 3, 1), (1, 2, 16, 127), (0, 1, 9, 64)):
        e = torch.zeros_like(x)
        e[b, h, n, c] = 4.0
        slope = (u.double() * (S.rope(e, r).double() - S.rope(-e, r).double())).sum() / 8.0
        # two outputs of size up to 4, rounded by 2^-8 of it at most, times u, over 4; the gradient rounded itself
        tol = 2.0 ** -8 * 2 * float(u[b, h, n].abs().max()) + float(leaf.grad[b, h, n, c].abs()) * 2.0 ** -8 + 1e-4
        assert abs(float(slope) - float(leaf.grad[b, h, n, c])) <= tol
    # on a stream of its own
    st = torch.cuda.Stream()
    leaf = x.clone().requires_grad_()
    torch.cuda.synchronize()
    y = S.rope(leaf, r, stream=st)
    st.synchronize()
    y.backward(u)
    torch.cuda.synchronize()
    assert torch.equal(y, S.rope(x, r)) and torch.equal(leaf.grad, S.rope(u, r, inverse=True))
    # positions changed in between: refused, as for any saved tensor
    start = T.i32([3, 4])
    y = S.rope(x.clone().requires_grad_(), r, start=start)
    start += 1
    with pytest.raises(RuntimeError, match="modified"):
        y.backward(u)
    # forward and backward in one graph, replayed with other values
    leaf, grad, start = x.clone().requires_grad_(), u.clone(), T.i32([0, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(S.rope(leaf, r, start=start), leaf, grad)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = S.rope(leaf, r, start=start)
        (dx,) = torch.autograd.grad(y, leaf, grad)
    for k in (7, 100000):
        grad.copy_(view(B, H, N, D, "nhd", seed=k))
        start.copy_(T.i32([k, 2 * k]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, S.rope(x, r, start=start)) and torch.equal(dx, S.rope(grad, r, start=start, inverse=True))
