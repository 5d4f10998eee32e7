// sage_paged_sched.cuh - how the paged attention kernels share their work.
//
// The work is a list of items.  An item is a set of up to M query rows of one
// key head and the key sequence they read, cut into tiles of TK keys.  The
// list holds, in this order,
//   (1) for each key head and each M rows of ALL requests' rows: the shared
//       prefix (only when the prefix is computed once for all: pre_rt > 0);
//   (2) for each request, key head and M rows of that request: its own keys,
//       preceded by the prefix when join = 1.
// The tiles of the list, numbered through, are cut into equal runs, one for
// each worker (a warp or a CTA).  So the split follows the lengths that the
// device holds: a long sequence is shared among many workers, several short
// ones fall to a single worker, and no host value depends on the lengths.
// A worker leaves a partial result (running maximum, sum and unnormalised
// output) for each item it touches, in slot worker + item: along the list
// either the worker or the item advances by one, so the slots are distinct.
#pragma once

#include "sage_paged.h"

namespace sage {

__device__ __forceinline__ int paged_clamp(const int32_t* lens, int b, int n) {
    if (lens == nullptr) return n;
    const int v = __ldg(lens + b);
    return v < 0 ? 0 : (v > n ? n : v);
}

template <int M, int TK>
struct PagedSched {
    // The 128-key lists' worker writes whole rows itself, so rows that see no
    // key have a tile too (with no visible key: zeros).
    static constexpr bool kWholeRows = TK == 128;
    const PagedParams& p;
    int lp;                              // prefix length
    __device__ explicit PagedSched(const PagedParams& pp) : p(pp) {
        lp = p.Wp > 0 ? paged_clamp(p.prefix_len, 0, p.Wp * p.page) : 0;
    }
    __device__ int q_rows(int b) const { return paged_clamp(p.q_len, b, p.Nq); }
    __device__ int own_keys(int b) const { return paged_clamp(p.kv_len, b, p.W * p.page); }
    __device__ int pre_tiles() const { return (lp + TK - 1) / TK; }
    __device__ int pre_total() const { return p.pre_rt * p.Hkv * pre_tiles(); }
    // own keys that some row of row tile rt sees (n query tokens, len own keys)
    __device__ int own_end(int n, int len, int rt) const {
        const int rows = n * p.G;
        if (rt * M >= rows) return 0;
        if (!p.causal) return len;
        const int last = (min(rt * M + M, rows) - 1) / p.G;
        return max(0, min(len, len - n + last + 1));
    }
    __device__ int item_tiles(int n, int len, int rt) const {
        if (rt * M >= n * p.G) return 0;
        const int nt = (own_end(n, len, rt) + TK - 1) / TK + (p.join ? pre_tiles() : 0);
        return kWholeRows ? max(nt, 1) : nt;
    }
    // tiles of one key head of request b
    __device__ int head_tiles(int b) const {
        const int n = q_rows(b), len = own_keys(b);
        if (p.rt == 1) return item_tiles(n, len, 0);
        int s = 0;
#pragma unroll 1
        for (int rt = 0; rt < p.rt; ++rt) s += item_tiles(n, len, rt);
        return s;
    }
    // tiles of one worker, given the length of the list
    __device__ int per_worker(int total) const { return max(1, (total + p.workers - 1) / p.workers); }
};

// A place in the list.  b = -1: a prefix item (rt counts its row tiles).
struct PagedPlace {
    int b, h, rt;
    int tile, ntiles;                    // tile of the item, tiles of the item
    int n, len;                          // the request's query tokens and own keys
    int item;                            // number of the item in the list
};

template <int M, int TK>
__device__ __forceinline__ void paged_enter(const PagedSched<M, TK>& s, PagedPlace& x) {
    const PagedParams& p = s.p;
    if (x.b < 0) {
        x.ntiles = s.pre_tiles();
        x.item = x.h * p.pre_rt + x.rt;
    } else {
        x.ntiles = s.item_tiles(x.n, x.len, x.rt);
        x.item = p.pre_rt * p.Hkv + (x.b * p.Hkv + x.h) * p.rt + x.rt;
    }
}

// The length of the list, and where the CTA's workers begin.  A block of
// THREADS threads sums the requests' tiles, thread t those of requests
// [t*cb, (t+1)*cb); the thread whose requests hold the first tile of worker
// first_worker + w*worker_step (w < NW) leaves {request, list position of its
// first tile} in found[w] ({-1, 0}: among the prefix items).  With `publish`
// the positions of all requests go to p.start as well.  `red` holds THREADS/32
// ints.  Ends with a barrier.
template <int M, int TK, int THREADS, int NW>
__device__ __forceinline__ int paged_scan(const PagedSched<M, TK>& s, int first_worker, int worker_step, int2* found,
                                          int* red, bool publish) {
    const PagedParams& p = s.p;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int cb = (p.B + THREADS - 1) / THREADS;
    const int b0 = min(t * cb, p.B), b1 = min(b0 + cb, p.B);
    int mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += s.head_tiles(b) * p.Hkv;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) red[w] = inc;
    if (t < NW) found[t] = make_int2(-1, 0);
    __syncthreads();
    int base = s.pre_total(), total = base;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < w) base += red[i];
        total += red[i];
    }
    base += inc - mine;
    const int per = s.per_worker(total);
    if (cb == 1 && !publish) {
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const int at = (first_worker + k * worker_step) * per;
            if (at >= base && at - base < mine) found[k] = make_int2(b0, base);
        }
    } else {
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int n = s.head_tiles(b) * p.Hkv;
#pragma unroll 1
            for (int k = 0; k < NW; ++k) {
                const int at = (first_worker + k * worker_step) * per;
                if (at >= base && at - base < n) found[k] = make_int2(b, base);
            }
            if (publish) p.start[b] = base;
            base += n;
        }
        if (publish && t == 0) p.start[p.B] = total;
    }
    __syncthreads();
    return total;
}

// The place of list position t (t < total), with paged_scan's finding.
template <int M, int TK>
__device__ __forceinline__ PagedPlace paged_place(const PagedSched<M, TK>& s, int2 found, int t) {
    const PagedParams& p = s.p;
    PagedPlace x{};
    x.b = found.x;
    if (x.b < 0) {
        const int nt = s.pre_tiles();
        x.item = t / nt;
        x.tile = t - x.item * nt;
        x.h = x.item / p.pre_rt;
        x.rt = x.item - x.h * p.pre_rt;
        x.ntiles = nt;
        return x;
    }
    x.n = s.q_rows(x.b);
    x.len = s.own_keys(x.b);
    int per_head = 0;
#pragma unroll 1
    for (int rt = 0; rt < p.rt; ++rt) per_head += s.item_tiles(x.n, x.len, rt);
    int at = t - found.y;
    x.h = at / per_head;
    at -= x.h * per_head;
#pragma unroll 1
    for (x.rt = 0; x.rt < p.rt; ++x.rt) {
        const int nt = s.item_tiles(x.n, x.len, x.rt);
        if (at < nt) break;
        at -= nt;
    }
    x.tile = at;
    paged_enter(s, x);
    return x;
}

// The next tile of the list (the caller knows that there is one).
template <int M, int TK>
__device__ __forceinline__ void paged_next(const PagedSched<M, TK>& s, PagedPlace& x) {
    const PagedParams& p = s.p;
    if (++x.tile < x.ntiles) return;
    x.tile = 0;
    do {
        if (x.b < 0) {
            if (++x.rt == p.pre_rt) {
                x.rt = 0;
                if (++x.h == p.Hkv) { x.h = 0; x.b = 0; x.n = s.q_rows(0); x.len = s.own_keys(0); }
            }
        } else if (++x.rt == p.rt) {
            x.rt = 0;
            if (++x.h == p.Hkv) {
                x.h = 0;
                if (++x.b >= p.B) { x.ntiles = 0; return; }
                x.n = s.q_rows(x.b);
                x.len = s.own_keys(x.b);
            }
        }
        paged_enter(s, x);
    } while (x.ntiles == 0);
}

// What a tile's keys are.
struct PagedSpan {
    bool own;                            // own keys of request b, else the prefix
    int key0;                            // first key, in its sequence
    int nkeys;                           // keys of the tile that exist (<= TK)
};
template <int M, int TK>
__device__ __forceinline__ PagedSpan paged_span(const PagedSched<M, TK>& s, const PagedPlace& x) {
    PagedSpan r;
    const int np = (x.b < 0 || s.p.join) ? s.pre_tiles() : 0;
    r.own = x.tile >= np;
    r.key0 = (r.own ? x.tile - np : x.tile) * TK;
    r.nkeys = min(TK, (r.own ? x.len : s.lp) - r.key0);
    return r;
}

// Row r of an item: its request, query token and query head (false: no such row).
template <int M, int TK>
__device__ __forceinline__ bool paged_row(const PagedSched<M, TK>& s, const PagedPlace& x, int r, int& b, int& i, int& hq) {
    const PagedParams& p = s.p;
    int row = x.rt * M + r;
    b = x.b;
    if (x.b < 0) {
        const int per = p.Nq * p.G;
        b = row / per;
        row -= b * per;
        if (b >= p.B) return false;
    }
    i = row / p.G;
    hq = x.h * p.G + (row - i * p.G);
    return i < (x.b < 0 ? s.q_rows(b) : x.n);
}

// 16 bytes to shared memory, the first `bytes` of them from src, zeros behind.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

}  // namespace sage
