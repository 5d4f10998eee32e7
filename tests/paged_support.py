"""Helpers of the page-cache tests: problems whose unused cache rows are NaN,
and the operators from their definition in 64 bits."""
from __future__ import annotations

import math
import random
from dataclasses import dataclass, field

import torch

import quantized_exact_attention_gb300 as S

U_BF16 = torch.finfo(torch.bfloat16).eps / 2      # one rounding to BF16, relative
U_F32 = torch.finfo(torch.float32).eps / 2


@dataclass
class Paged:
    """One attention problem; every tensor on `device`."""
    q: torch.Tensor
    cache_k: torch.Tensor
    cache_v: torch.Tensor
    table: torch.Tensor | None
    q_len: list
    kv_len: list
    prefix_table: torch.Tensor | None
    prefix_len: int
    causal: bool
    sm_scale: float = 0.0
    extra: dict = field(default_factory=dict)


def make(B, H, Hkv, D, Nq, page, q_len=None, kv_len=None, prefix=0, causal=True, seed=0, device="cuda",
         layout="nhd", spare=3, table_pad=2, scale=1.0, sm_scale=0.0, poison=float("nan")) -> Paged:
    """Random problem: pages in random order, rows that no request holds are
    `poison`, table entries behind a length are far outside the cache."""
    g = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    q_len = [Nq] * B if q_len is None else list(q_len)
    kv_len = [Nq] * B if kv_len is None else list(kv_len)
    need = [-(-n // page) for n in kv_len]
    pre = -(-prefix // page)
    pages = list(range(sum(need) + pre + spare))
    r.shuffle(pages)
    n_pages = len(pages)
    k = torch.full((n_pages, page, Hkv, D), poison, dtype=torch.bfloat16)
    v = torch.full((n_pages, page, Hkv, D), poison, dtype=torch.bfloat16)

    def fill(page_list, n):
        for j, pg in enumerate(page_list):
            m = min(page, n - j * page)
            k[pg, :m] = (torch.randn((m, Hkv, D), generator=g) * scale).to(torch.bfloat16)
            v[pg, :m] = torch.randn((m, Hkv, D), generator=g).to(torch.bfloat16)

    ptable = None
    if prefix:
        lst = [pages.pop() for _ in range(pre)]
        fill(lst, prefix)
        ptable = torch.tensor(lst + [n_pages + 5] * table_pad, dtype=torch.int32)
    W = max(need + [1]) + table_pad
    table = torch.full((B, W), n_pages + 7, dtype=torch.int32)
    for b in range(B):
        lst = [pages.pop() for _ in range(need[b])]
        fill(lst, kv_len[b])
        table[b, :len(lst)] = torch.tensor(lst, dtype=torch.int32)
    q = torch.randn((B, H, Nq, D), generator=g).to(torch.bfloat16)
    if layout == "nhd":
        q = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        ck, cv = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    else:                                                   # pages head by head, K and V interleaved in one buffer
        kv = torch.stack((k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)), 1).contiguous().to(device)
        ck, cv = kv[:, 0], kv[:, 1]
    mv = lambda t: t.to(device) if t is not None else None  # noqa: E731
    return Paged(mv(q), mv(ck), mv(cv), mv(table), q_len, kv_len, mv(ptable), prefix, causal, sm_scale)


def reference(p: Paged):
    """(output, tolerance) in float64, from the definition.

    The tolerance follows the roundings the kernels make, per element:
    with A = sum_j w_j |v_j| (normalised weights w),
      - the weights rounded to BF16:             U_BF16 * A
      - the weights' own error delta, in the numerator and in the sum: 2 delta A
      - the output rounded to BF16:              U_BF16 * |o + errors above|
    delta covers the FP32 scores (a dot product of D exact products, each
    addition off by at most 2 U_F32 of the partial sums' bound sum |q k|, also
    where the adder truncates), their scaling and difference to the maximum
    (4 U_F32 |s|), and the exponential and the joins (2^-20, several ulp).
    """
    B, H, N, D = p.q.shape
    heads, page = p.cache_k.shape[1], p.cache_k.shape[2]
    G = H // heads
    scale = p.sm_scale if p.sm_scale > 0 else 1.0 / math.sqrt(D)
    dev = p.q.device
    out = torch.zeros((B, H, N, D), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    for b in range(B):
        n, m = p.q_len[b], p.kv_len[b]
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
            if not ks or n == 0:
                continue
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            hidden = torch.zeros((n, k.shape[0]), dtype=torch.bool, device=dev)
            if p.causal and m:
                i, j = torch.arange(n, device=dev)[:, None], torch.arange(m, device=dev)[None]
                hidden[:, p.prefix_len:] = j > i + (m - n)
            q = p.q[b, h * G:(h + 1) * G, :n].double()
            s = q @ k.T * scale
            s = s.masked_fill(hidden, -math.inf)
            top = s.amax(-1, keepdim=True)
            w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            tot = w.sum(-1, keepdim=True)
            w = torch.where(tot > 0, w / tot, 0.0)
            o, A = w @ v, w @ v.abs()
            size = ((q.abs() @ k.abs().T) * scale).amax(-1, keepdim=True)
            delta = D * 2 * U_F32 * size + 4 * U_F32 * size + 2.0 ** -20
            err = (U_BF16 + 2 * delta) * A
            out[b, h * G:(h + 1) * G, :n] = o
            tol[b, h * G:(h + 1) * G, :n] = (err + U_BF16 * (o.abs() + err)) * 1.0001 + 1e-37
    return out, tol


def run(p: Paged, fill=None, lens_on_device=True, workspace=None, stream=None, o=None):
    """The library's result for p, into an output pre-filled with `fill`."""
    B, H, N, D = p.q.shape
    dev = p.q.device
    cache = S.PageCache(p.cache_k, p.cache_v)
    if o is None:
        o = torch.full((B, N, H, D), 7.0 if fill is None else fill, dtype=torch.bfloat16, device=dev).permute(0, 2, 1, 3)
    if workspace is None:
        workspace = S.alloc_paged_workspace(B, H, cache.heads, N, D, dev)
        workspace.fill_(0xFF)                               # every float of it NaN
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    S.sage_attn_paged(p.q, o, cache, p.table, workspace, q_len=i32(p.q_len), kv_len=i32(p.kv_len),
                      prefix_table=p.prefix_table, prefix_len=i32([p.prefix_len]) if p.prefix_table is not None else None,
                      sm_scale=p.sm_scale, causal=p.causal, stream=stream)
    return o


def check(p: Paged, o, fill=7.0):
    """o against the definition; rows at or beyond q_len still hold `fill`."""
    torch.cuda.synchronize()
    assert S.sage_get_device_status() == S.SAGE_OK
    ref, tol = reference(p)
    for b, n in enumerate(p.q_len):
        assert bool((o[b, :, n:] == fill).all()), f"rows behind q_len of request {b} were written"
        d = (o[b, :, :n].double() - ref[b, :, :n]).abs()
        bad = ~(d <= tol[b, :, :n])
        assert not bool(bad.any()), (
            f"request {b}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {bad.nonzero()[0].tolist()}, "
            f"largest ratio {float((d / tol[b, :, :n]).nan_to_num(nan=float('inf')).max()):.3g}")


def tables_reference(old, new, page, free, table, n_slots):
    """Lists (table, slots, taken) from the definition."""
    B, W = len(new), len(table[0])
    cap = W * page
    out, slots, taken = [], [], 0
    for b in range(B):
        a = min(max(old[b], 0), cap)
        n = max(a, min(max(new[b], 0), cap))
        pa, pn = -(-a // page), -(-n // page)
        row = list(table[b][:pa])
        for _ in range(pa, pn):
            row.append(free[taken] if taken < len(free) else -1)
            taken += 1
        row += [-1] * (W - len(row))
        out.append(row)
        sl = []
        for i in range(n_slots):
            t = a + i
            s = -1
            if t < n and row[t // page] >= 0:
                s = row[t // page] * page + t % page
            sl.append(s if s <= 2 ** 31 - 1 else -1)
        slots.append(sl)
    return out, slots, taken
