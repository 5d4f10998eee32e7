// sage_paged_sched.cuh - how the paged attention kernels share their work.
//
// The work is a list of items.  An item is a set of query rows of one key head
// and the key sequence they read, cut into tiles of TK keys.  The list holds
//   for a prefix computed once for all (pre_rt > 0; tiles kernel only): for
//   each set of rows out of ALL requests' rows, and each key head, the shared
//   prefix;
//   then, for each request, each set of its rows (rt > 0), and each key head:
//   its own keys, preceded by the prefix when join = 1.
// Each item takes as many places in the list as it has tiles, and kItemCost in
// front of them, which stand for what an item costs a worker besides its tiles
// (fetching its rows, writing its output).  The places are cut into equal
// runs, one for each worker (a warp or a CTA).  So the split follows the lengths
// that the device holds: a long sequence is shared among many workers, several
// short ones fall to a single worker, and no host value depends on the lengths.
// Runs have a least length.  Tiles: kItemCost, as a shorter run costs more at
// its ends than it saves (64 requests behind 2,048 shared keys, runs of 1 place:
// 51 us, 3: 43.7, 6: 46.4).  Few rows: a run of r places of an item of T takes r
// steps and leaves T / r parts to join, which is least at r = sqrt(kPartCost T)
// (one key head, 12,000 keys, 1 place: 21.3 us, 6: 12.0; 40,000 keys, 3: 24.4,
// 8: 17.7; but items of 2 steps, 1: 9.6, 6: 11.4).
// A worker leaves a partial result (running maximum, sum and unnormalised
// output) for an item it shares, in slot worker + item (the prefix's items and
// the others are numbered and kept apart): along the list either the worker or
// the item advances by one, so the slots are distinct.
//
// Sets of rows, in the order of query token, then query head of the key head:
//   few-rows kernel (TK = 16): M rows after one another;
//   many-rows kernel (TK = 128): groups of 128 rows that hold `tok` whole tokens
//   (of the shared prefix's items: `pre_tok` whole requests), so that a group is
//   one box of a tensor map; the rows left over stay empty.
#pragma once

#include "sage_paged.h"

namespace sage {

__device__ __forceinline__ int paged_clamp(const int32_t* lens, int b, int n, bool early) {
    if (lens == nullptr) return n;
    const int v = early ? ld_gpu(lens + b) : lens[b];
    return v < 0 ? 0 : (v > n ? n : v);
}

// n / d for 0 <= n < 2^31 (FastDiv, made by the host).
__device__ __forceinline__ int fast_div(int n, const FastDiv& f) {
    return (int)((__umulhi((uint32_t)n, f.m) + (uint32_t)n) >> f.s);
}

// n / d for 0 <= n < 2^30, 0 < d, and a quotient below 2^20, which the
// approximation misses by one at most.
__device__ __forceinline__ int small_div(int n, int d) {
    const int q = (int)__fdividef((float)n, (float)d), r = n - q * d;
    return q + (r >= d ? 1 : 0) - (r < 0 ? 1 : 0);
}

// kPre: the list holds items of the shared prefix.
template <int M, int TK, bool kPre>
struct PagedSched {
    static constexpr bool kTiles = TK == 128;
    static constexpr int kItemCost = kTiles ? 3 : 1;
    static constexpr float kPartCost = 0.04f;             // joining a part, in places
    const PagedParams& p;
    bool early;                          // the lengths are read before the kernel's own pdl_wait, without a fence
    int lp;                              // prefix length
    __device__ explicit PagedSched(const PagedParams& pp, bool before_wait = false) : p(pp), early(before_wait) {
        lp = p.Wp > 0 ? paged_clamp(p.prefix_len, 0, p.Wp * p.page, early) : 0;
    }
    __device__ int q_rows(int b) const { return paged_clamp(p.q_len, b, p.Nq, early); }
    __device__ int own_keys(int b) const { return paged_clamp(p.kv_len, b, p.W * p.page, early); }
    __device__ int pre_tiles() const { return (lp + TK - 1) / TK; }
    // places of an item of nt tiles
    __device__ static int places(int nt) { return nt > 0 ? nt + kItemCost : 0; }
    // Places of each of `workers` runs of a list of `total` places, `items` items.
    __device__ static int share(int total, const FastDiv& workers, int count, int items) {
        const int least = kTiles ? kItemCost : 1 + (int)sqrtf(kPartCost * (float)total / (float)items);
        return max(least, fast_div(total + count - 1, workers));
    }
    __device__ int pre_total() const { return kPre ? p.pre_rt * p.Hkv * places(pre_tiles()) : 0; }
    // Tiles of row set rt of a request with n query tokens and len own keys.
    __device__ int item_tiles(int n, int len, int rt) const {
        int last;                        // last token of the set that exists
        if constexpr (kTiles) {
            const int toks = p.tok * (M / 128);
            if (rt * toks >= n) return 0;
            last = min((rt + 1) * toks, n) - 1;
        } else {
            if (rt * M >= n * p.G) return 0;
            last = rt + 1 == p.rt ? n - 1 : min(fast_div(rt * M + M - 1, p.by_G), n - 1);
        }
        const int end = p.causal ? max(0, min(len, len - n + last + 1)) : len;      // own keys that some row sees
        const int nt = (end + TK - 1) / TK + (p.join ? pre_tiles() : 0);
        // the tiles kernel writes whole rows itself unless the prefix's parts
        // are still to come, so rows that see no key have a tile too (with no
        // visible key: zeros)
        return kTiles && !kPre ? max(nt, 1) : nt;
    }
};

// The length of the list, and where the CTA's workers begin.  A block of
// THREADS threads sums the places of the (request, row set) pairs; the thread
// whose pairs hold the first place of worker first_worker + w*worker_step
// (w < NW) leaves {pair, the pair's first place} in found[w] ({-1, 0}: a
// list of prefix items).  With `publish` the positions of all
// pairs go to p.start as well.  `red` holds THREADS/32 ints.  Ends with a
// barrier.
template <int M, int TK, bool kPre, int THREADS, int NW>
__device__ __forceinline__ int paged_scan(const PagedSched<M, TK, kPre>& s, int first_worker, int worker_step, int2* found,
                                          int* red, bool publish) {
    const PagedParams& p = s.p;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int pairs = p.B * p.rt, cb = (pairs + THREADS - 1) / THREADS;
    const int u0 = min(t * cb, pairs), u1 = min(u0 + cb, pairs);
    const int b0 = p.rt > 1 ? fast_div(u0, p.by_rt) : u0;
    int mine = 0;
    {
        int b = b0, rt = u0 - b0 * p.rt;
#pragma unroll 1
        for (int u = u0; u < u1; ++u) {
            mine += s.places(s.item_tiles(s.q_rows(b), s.own_keys(b), rt)) * p.Hkv;
            if (++rt == p.rt) { rt = 0; ++b; }
        }
    }
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
    const int per = s.share(total, p.by_workers, p.workers, pairs * p.Hkv);
    int b = b0, rt = u0 - b0 * p.rt;
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
        const int n = cb == 1 ? mine : s.places(s.item_tiles(s.q_rows(b), s.own_keys(b), rt)) * p.Hkv;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const int at = (first_worker + k * worker_step) * per;
            if (at >= base && at - base < n) found[k] = make_int2(u, base);
        }
        if (publish) p.start[u] = base;
        base += n;
        if (++rt == p.rt) { rt = 0; ++b; }
    }
    if (publish && t == 0) p.start[pairs] = total;
    __syncthreads();
    return total;
}

// A tile in the list.  b = -1: a prefix item (rt counts its row sets).
struct PagedPlace {
    int b, h, rt;
    int tile, ntiles;                    // tile of the item, tiles of the item
    int n, len;                          // the request's query tokens and own keys
    int item;                            // number of the item in the list
    int pos;                             // the tile's place
};

// The first tile at or behind place t (t < total), with paged_scan's finding.
template <int M, int TK, bool kPre>
__device__ __forceinline__ PagedPlace paged_place(const PagedSched<M, TK, kPre>& s, int2 found, int t) {
    const PagedParams& p = s.p;
    PagedPlace x{};
    int o;                               // place within the item
    if (kPre && found.x < 0) {
        x.b = -1;
        x.ntiles = s.pre_tiles();
        x.item = t / s.places(x.ntiles);
        o = t - x.item * s.places(x.ntiles);
        x.rt = x.item / p.Hkv;
        x.h = x.item - x.rt * p.Hkv;
    } else {
        x.b = p.rt > 1 ? fast_div(found.x, p.by_rt) : found.x;
        x.rt = found.x - x.b * p.rt;
        x.n = s.q_rows(x.b);
        x.len = s.own_keys(x.b);
        x.ntiles = s.item_tiles(x.n, x.len, x.rt);
        x.h = small_div(t - found.y, s.places(x.ntiles));
        o = t - found.y - x.h * s.places(x.ntiles);
        x.item = found.x * p.Hkv + x.h;
    }
    x.tile = max(0, o - s.kItemCost);
    x.pos = t - o + s.kItemCost + x.tile;
    return x;
}

// The next tile of the list (its place is behind the list when there is none).
template <int M, int TK, bool kPre>
__device__ __forceinline__ void paged_next(const PagedSched<M, TK, kPre>& s, PagedPlace& x) {
    const PagedParams& p = s.p;
    ++x.pos;
    if (++x.tile < x.ntiles) return;
    x.pos += s.kItemCost;
    x.tile = 0;
    ++x.item;
    if (++x.h < p.Hkv) return;
    x.h = 0;
    ++x.rt;
    if (kPre && x.b < 0) {
        if (x.rt < p.pre_rt) return;
        x.item = 0;
        x.rt = p.rt;                     // behind request -1
    }
    for (;; ++x.rt, x.item += p.Hkv) {   // the next row set that has tiles
        if (x.rt == p.rt) {
            x.rt = 0;
            if (++x.b >= p.B || (kPre && p.rt == 0)) { x.ntiles = 0; x.pos = INT32_MAX; return; }
            x.n = s.q_rows(x.b);
            x.len = s.own_keys(x.b);
        }
        x.ntiles = s.item_tiles(x.n, x.len, x.rt);
        if (x.ntiles > 0) return;
    }
}

// What a tile's keys are.
struct PagedSpan {
    bool own;                            // own keys of request b, else the prefix
    int key0;                            // first key, in its sequence
    int nkeys;                           // keys of the tile that exist (<= TK; 0 in an item without keys)
};
template <int M, int TK, bool kPre>
__device__ __forceinline__ PagedSpan paged_span(const PagedSched<M, TK, kPre>& s, int b, int len, int tile) {
    PagedSpan r;
    const bool pre = kPre && b < 0;
    const int np = pre || s.p.join ? s.pre_tiles() : 0;
    r.own = !pre && tile >= np;
    r.key0 = (r.own ? tile - np : tile) * TK;
    r.nkeys = min(TK, (r.own ? len : s.lp) - r.key0);
    return r;
}

// Row r of an item: its request, query token and query head (false: no such
// row).  n: query tokens of the item's request.
template <int M, int TK, bool kPre>
__device__ __forceinline__ bool paged_row(const PagedSched<M, TK, kPre>& s, int ib, int ih, int irt, int n, int r, int& b, int& i,
                                          int& hq) {
    const PagedParams& p = s.p;
    if constexpr (PagedSched<M, TK, kPre>::kTiles) {
        const int group = irt * (M / 128) + (r >> 7);
        int rr = r & 127;
        if (kPre && ib < 0) {
            const int u = fast_div(rr, p.by_pre_unit);
            rr -= u * p.pre_unit;
            b = group * p.pre_tok + u;
            i = fast_div(rr, p.by_G);
            hq = ih * p.G + rr - i * p.G;
            return u < p.pre_tok && b < p.B && i < s.q_rows(b);
        }
        const int u = fast_div(rr, p.by_G);
        b = ib;
        i = group * p.tok + u;
        hq = ih * p.G + rr - u * p.G;
        return u < p.tok && i < n;
    } else {
        const int row = irt * M + r;
        b = ib;
        i = fast_div(row, p.by_G);
        hq = ih * p.G + row - i * p.G;
        return i < n;
    }
}

// 16 bytes to shared memory, the first `bytes` of them from src, zeros behind.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

}  // namespace sage
