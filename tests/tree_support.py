"""Helpers of the tests of rotary positions and of trees of drafted tokens: the
operators from their definition in 64 bits."""
from __future__ import annotations

import math
import random
from fractions import Fraction

import torch

import quantized_exact_attention_gb300 as S
from tests import paged_support as P

# 2 pi to 60 digits
TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


def i32(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def angles(positions, frequencies, device="cuda"):
    """positions [B, N] (ints) times frequencies, modulo 2 pi, in float64 [B, N, R / 2]: exact in between."""
    fr = [Fraction(f) for f in frequencies]
    known = {}
    for p in {int(p) for row in positions for p in row}:
        known[p] = [float(x - TWO_PI * math.floor(x / TWO_PI)) for x in (p * f for f in fr)]
    return torch.tensor([[known[int(p)] for p in row] for row in positions], dtype=torch.float64, device=device)


def turned(x, angle, rotary_dim, interleaved, amplitude=1.0, inverse=False):
    """(x rotated, bound of what the kernel may be off by before its one rounding to BF16), float64 [B, H, N, D].

    The kernel's cosine and sine: an angle x of up to pi / 4 in FP32, three roundings (3 * 2^-24 x, times the slope:
    1.0e-7), cut at 2^-32 turns (2e-9); a Taylor series (3e-8) summed in FP32 (4e-8); the amplitude's product (2^-24): below
    2.8e-7 together.  The two products and their sum in FP32: 2^-24 of each once more for the product and once for the sum,
    below 1.2e-7 of |x1| + |x2|.  Together below 2^-21 A (|x1| + |x2|)."""
    R, half = rotary_dim, rotary_dim // 2
    x = x.double()
    c, s = amplitude * torch.cos(angle)[:, None], amplitude * torch.sin(angle)[:, None]
    if inverse:
        s = -s
    first = torch.tensor([2 * j if interleaved else j for j in range(half)], device=x.device)
    second = first + (1 if interleaved else half)
    a, b = x[..., first], x[..., second]
    y, off = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    off[..., first] = off[..., second] = 2.0 ** -21 * abs(amplitude) * (a.abs() + b.abs())
    return y, off


def near(got, want, off):
    """got (BF16) within `off` and one rounding of want."""
    tol = off + P.U_BF16 * (want.abs() + off)
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} outside the bound, first at "
                                 f"{bad.nonzero()[0].tolist()}")


def sees_of(parents):
    """For each token of one tree the set of tokens it sees."""
    out = []
    for i, p in enumerate(parents):
        out.append({i} | (out[p] if 0 <= p < i else set()))
    return out


def random_parents(r: random.Random, N, deep):
    """Parents of N tokens: a chain with deep = 0, else each follows one of the `deep` tokens before it, or none."""
    if deep == 0:
        return list(range(-1, N - 1))
    return [-1 if i == 0 or r.random() < 0.05 else r.randrange(max(0, i - deep), i) for i in range(N)]


def words_of(sees, N, width=None):
    """int32 words [N][width] of a list of sets."""
    width = -(-N // 32) if width is None else width
    rows = []
    for s in sees:
        row = [0] * width
        for t in s:
            row[t // 32] |= 1 << (t % 32)
        rows.append([w - (1 << 32) if w >> 31 else w for w in row])
    return rows


def reference(p: P.Paged, sees):
    """(output, tolerance) of the attention with sees[b][i] = the new tokens row i of request b sees, in float64; the
    roundings are those of paged_support.reference."""
    B, H, N, D = p.q.shape
    heads, page = p.cache_k.shape[1], p.cache_k.shape[2]
    G = H // heads
    scale = p.sm_scale if p.sm_scale > 0 else 1.0 / math.sqrt(D)
    dev = p.q.device
    out = torch.zeros((B, H, N, D), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    for b in range(B):
        n, m = p.q_len[b], p.kv_len[b]
        if n == 0 or (m == 0 and not p.prefix_len):
            continue
        visible = torch.ones((n, p.prefix_len + m), dtype=torch.bool)
        for i in range(n):
            for t in range(n):
                j = m - n + t
                if j >= 0 and t not in sees[b][i]:
                    visible[i, p.prefix_len + j] = False
        visible = visible.to(dev)
        pages = p.table[b, :-(-m // page)].long() if m else None
        for h in range(heads):
            ks, vs = [], []
            if p.prefix_len:
                pt = p.prefix_table[:-(-p.prefix_len // page)].long()
                ks.append(p.cache_k[pt, h].reshape(-1, D)[:p.prefix_len])
                vs.append(p.cache_v[pt, h].reshape(-1, D)[:p.prefix_len])
            if m:
                ks.append(p.cache_k[pages, h].reshape(-1, D)[:m])
                vs.append(p.cache_v[pages, h].reshape(-1, D)[:m])
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            q = p.q[b, h * G:(h + 1) * G, :n].double()
            s = (q @ k.T * scale).masked_fill(~visible, -math.inf)
            top = s.amax(-1, keepdim=True)
            w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            tot = w.sum(-1, keepdim=True)
            w = torch.where(tot > 0, w / tot, 0.0)
            o, A = w @ v, w @ v.abs()
            size = ((q.abs() @ k.abs().T) * scale).amax(-1, keepdim=True)
            delta = D * 2 * P.U_F32 * size + 4 * P.U_F32 * size + 2.0 ** -20
            err = (P.U_BF16 + 2 * delta) * A
            out[b, h * G:(h + 1) * G, :n] = o
            tol[b, h * G:(h + 1) * G, :n] = (err + P.U_BF16 * (o.abs() + err)) * 1.0001 + 1e-37
    return out, tol


def run(p: P.Paged, mask, fill=7.0, workspace=None, stream=None, o=None):
    """The library's result for p with this mask, into an output pre-filled with `fill`."""
    B, H, N, D = p.q.shape
    cache = S.PageCache(p.cache_k, p.cache_v)
    if o is None:
        o = torch.full((B, N, H, D), fill, dtype=torch.bfloat16, device=p.q.device).permute(0, 2, 1, 3)
    if workspace is None:
        workspace = S.alloc_paged_workspace(B, H, cache.heads, N, D, p.q.device)
        workspace.fill_(0xFF)                               # every float of it NaN
    S.sage_attn_paged_tree(p.q, o, cache, p.table, mask, workspace, q_len=i32(p.q_len), kv_len=i32(p.kv_len),
                           prefix_table=p.prefix_table, prefix_len=i32([p.prefix_len]) if p.prefix_table is not None else None,
                           sm_scale=p.sm_scale, stream=stream)
    return o


def check(p: P.Paged, sees, o, fill=7.0):
    """o against the definition; rows at or beyond q_len still hold `fill`."""
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    ref, tol = reference(p, sees)
    for b, n in enumerate(p.q_len):
        assert bool((o[b, :, n:] == fill).all()), f"rows behind q_len of request {b} were written"
        d = (o[b, :, :n].double() - ref[b, :, :n]).abs()
        bad = ~(d <= tol[b, :, :n])
        assert not bool(bad.any()), (f"request {b}: {int(bad.sum())} of {bad.numel()} outside the bound, first at "
                                     f"{bad.nonzero()[0].tolist()}")


def keep_reference(kept, slots, rows):
    """rows: dict slot -> value, moved request by request in the order of the entries."""
    for path, at in zip(kept, slots):
        for i, t in enumerate(path):
            if 0 <= t < len(at) and at[t] >= 0 and at[i] >= 0:
                rows[at[i]] = rows[at[t]]
    return rows
