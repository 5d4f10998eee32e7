// sage_tree.cu - bookkeeping of a tree of drafted tokens on the GPU: which
// tokens each of them sees, from the tree's parents, and the move of the
// accepted tokens' cache rows to the front.
#include <algorithm>

#include "sage_gb300.h"
#include "sage_internal.h"
#include "sage_paged.h"

namespace sage {
namespace {

// ---------------------------------------------------------------------------
// Tree tables: see(i) = {i} u see(parent(i)), depth(i) = |see(i)| - 1.
//
// Parents come before their children.  A warp takes 32 tokens, whose bits make
// one word, and finds for each of them its ancestors among the 32 by doubling
// (five rounds of shuffles), and the first ancestor before them, the parent of
// the lowest one found.  Then a thread goes through its row's words from the
// last to the first: a word is that of the ancestor it has come to, or 0; so a
// row takes as many steps as it has words, however deep the tree is (a walk
// from parent to parent, 1,024 trees of 250 tokens, 22 levels: 6.3 us, so 5.3).
// A block holds the words of its tokens and those before them in shared memory:
// of several requests where trees are small.  A row's words leave through shared
// memory, a sector of 32 bytes at a time (each thread writing its own: 11.6 us in
// place of 6.3).
// ---------------------------------------------------------------------------
constexpr int kTreeThreads = 256;
constexpr int kTreeTokens = 4096;        // of a request, at most: a block holds 8 bytes of each
constexpr int kStageWords = 8;           // words of a row that leave together

struct TreeParams {
    const int32_t* parents;
    const int32_t* n_len;                // or null: N
    int32_t* mask;
    int32_t* depth;                      // or null
    int64_t psb, msb, msn, dsb;
    int B, N, W;
    int pack;                            // requests of a block, W warps each (1: a block takes 256 tokens of one)
};

// kHeld: tokens that a block holds.
template <int kHeld>
__global__ void __launch_bounds__(kTreeThreads) tree_tables_kernel(const __grid_constant__ TreeParams p) {
    constexpr int kWarps = kTreeThreads / 32;
    __shared__ int2 held[kHeld];                           // a token's word of its own 32, its first ancestor before them
    __shared__ uint32_t stage[kWarps][32][kStageWords + 1];
    pdl_trigger();
    pdl_wait();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    int b, i, base = 0;                                    // base: of the request's tokens in `held`
    if (p.pack > 1) {
        const int r = warp / p.W;
        b = r < p.pack ? (int)blockIdx.x * p.pack + r : p.B;
        i = t - r * p.W * 32;
        base = r * p.W * 32;
    } else {
        b = blockIdx.x;
        i = (int)blockIdx.y * kTreeThreads + t;
    }
    const bool row = b < p.B && i < p.N;
    const int n = row && p.n_len != nullptr ? p.n_len[b] : p.N;
    auto hold = [&](int j) {                               // token j of request b, one of 32 after one another
        const int x = b < p.B && j < p.N ? p.parents[b * p.psb + j] : -1, j0 = j - lane;
        const int before = x < j ? x : -1;                 // a token whose parent is not one before it has none
        int up = before >= j0 ? before - j0 : -1;
        uint32_t bits = 1u << lane;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const int from = up < 0 ? lane : up;
            const uint32_t more = __shfl_sync(0xffffffffu, bits, from);
            const int next = __shfl_sync(0xffffffffu, up, from);
            if (up >= 0) {
                bits |= more;
                up = next;
            }
        }
        const int leaves = __shfl_sync(0xffffffffu, before, __ffs((int)bits) - 1);
        held[base + j] = make_int2((int)bits, leaves);
    };
    if (p.pack > 1) {
        if (b < p.B) hold(i);
    } else {
        const int last = min(p.N, ((int)blockIdx.y + 1) * kTreeThreads);
        for (int j = t; j - lane < last; j += kTreeThreads) hold(j);
    }
    __syncthreads();
    const int64_t m = row ? b * p.msb + i * p.msn : -1;
    int at = row && i < n ? i : -1, seen = 0;
    uint32_t(&mine)[32][kStageWords + 1] = stage[warp];
#pragma unroll 1
    for (int w0 = (p.W - 1) / kStageWords * kStageWords; w0 >= 0; w0 -= kStageWords) {
#pragma unroll 1
        for (int w = min(w0 + kStageWords, p.W) - 1; w >= w0; --w) {
            uint32_t bits = 0;
            if (at >= 32 * w) {
                const int2 x = held[base + at];
                bits = (uint32_t)x.x;
                at = x.y;
                seen += __popc(bits);
            }
            mine[lane][w - w0] = bits;
        }
        __syncwarp();
        // kStageWords lanes write a row's words
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 32 / kStageWords) {
            const int r = r0 + lane / kStageWords, w = lane % kStageWords;
            const int64_t to = __shfl_sync(0xffffffffu, m, r);
            if (to >= 0 && w0 + w < p.W) p.mask[to + w0 + w] = (int32_t)mine[r][w];
        }
        __syncwarp();
    }
    if (row && p.depth != nullptr) p.depth[b * p.dsb + i] = max(seen - 1, 0);
}

// ---------------------------------------------------------------------------
// Keep: the rows of token kept[b][i] move to the place of token i, for
// i = 0, 1, ... in order.  A thread moves one 16-byte column of K and of V
// through the moves of its request, so with one group of threads the order holds
// without a barrier.  A move reads what one before it wrote only where kept[b][i]
// < i, which an accepted path, ascending, never has; then the moves of the 32 go
// one by one.  Else no move reads what an earlier one writes, and six are in
// flight at a time, or four groups take every fourth of 32, all loaded before the
// first is stored (a later window reads nothing that an earlier one writes
// either, so one barrier a window does).
// Bound by HBM behind dependent loads (512 requests, 16 heads of 128 channels, up
// to 20 kept of 61, 82 MB: 16.5 us, 0.73 of the copy rate; with up to 6 kept, 21
// MB, 4.4 us; slots asked for behind the entries 16.8 and 4.6, with four in flight
// 5.3, and 5.8 where a thread has a column of either K or V and looks at all
// entries, eight in flight).
// ---------------------------------------------------------------------------
struct KeepParams {
    const int32_t* kept;
    const int32_t* slots;
    uint16_t* ck;
    uint16_t* cv;
    int* status;
    int64_t kept_stride, slots_stride, capacity;
    int64_t ckp, ckh, ckt, cvp, cvh, cvt;
    int N, K, columns, chunk_shift;      // columns: 16-byte columns of a token's K rows
    int page, page_shift;
};

constexpr int kKeepColumns = 64;         // of a block

template <int kGroups>
__global__ void __launch_bounds__(kKeepColumns * kGroups) cache_keep_kernel(const __grid_constant__ KeepParams p) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const int group = threadIdx.x / kKeepColumns, col = (int)blockIdx.y * kKeepColumns + threadIdx.x % kKeepColumns;
    const bool live = col < p.columns;
    const int h = col >> p.chunk_shift, c = (col - (h << p.chunk_shift)) * 8;
    uint16_t* k = p.ck + h * p.ckh + c;
    uint16_t* v = p.cv + h * p.cvh + c;
    const int32_t* slots = p.slots + b * p.slots_stride;
    auto row = [&](uint16_t* base, int slot, int64_t sp, int64_t st) -> uint4* {
        return reinterpret_cast<uint4*>(base + (int64_t)(slot >> p.page_shift) * sp + (int64_t)(slot & (p.page - 1)) * st);
    };
    // up to 64 slots are asked for beside the entries that name them
    const bool held = p.N <= 64;
    int slot0 = -1, slot1 = -1;
    if (held) {
        if (lane < p.N) slot0 = slots[lane];
        if (lane + 32 < p.N) slot1 = slots[lane + 32];
    }
#pragma unroll 1
    for (int i0 = 0; i0 < p.K; i0 += 32) {                 // a lane looks one move up
        const int i = i0 + lane;
        int src = -1, dst = -1, t = i < p.K ? p.kept[b * p.kept_stride + i] : -1;
        const bool names = t >= 0 && t < p.N && t != i;
        if (held) {
            const int lower = __shfl_sync(0xffffffffu, slot0, t & 31), upper = __shfl_sync(0xffffffffu, slot1, t & 31);
            if (names) {
                src = t < 32 ? lower : upper;
                dst = i0 == 0 ? slot0 : slot1;
            }
        } else if (names) {
            src = slots[t];
            dst = slots[i];
        }
        for (int s : {src, dst})
            if (s >= p.capacity && atomicCAS(p.status, 0, kErrPage) == 0) p.status[3] = s >> p.page_shift;
        const bool moves = src >= 0 && dst >= 0 && src < p.capacity && dst < p.capacity;
        uint32_t left = __ballot_sync(0xffffffffu, moves);
        const bool in_turn = __any_sync(0xffffffffu, moves && t < i);      // the same in every warp
        constexpr int kFlight = kGroups == 1 ? 6 : 32 / kGroups;
        uint4 x[kFlight], y[kFlight];
        int to[kFlight];
        if (kGroups == 1 || in_turn) {                     // the next moves that are left, by the first group
            if (kGroups > 1) __syncthreads();
            const int flight = in_turn ? 1 : kFlight;
#pragma unroll 1
            while (left != 0) {
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    const bool one = left != 0 && u < flight;
                    const int from = one ? __ffs((int)left) - 1 : 0;
                    const int s = __shfl_sync(0xffffffffu, src, from), d = __shfl_sync(0xffffffffu, dst, from);
                    to[u] = one && live && group == 0 ? d : -1;
                    if (one) left &= left - 1;
                    if (to[u] >= 0) {
                        x[u] = *row(k, s, p.ckp, p.ckt);
                        y[u] = *row(v, s, p.cvp, p.cvt);
                    }
                }
#pragma unroll
                for (int u = 0; u < kFlight; ++u)
                    if (to[u] >= 0) {
                        *row(k, to[u], p.ckp, p.ckt) = x[u];
                        *row(v, to[u], p.cvp, p.cvt) = y[u];
                    }
            }
            if (kGroups > 1) __syncthreads();
        } else {                                           // a group takes every kGroups-th entry
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const int from = u * kGroups + group;
                const int s = __shfl_sync(0xffffffffu, src, from), d = __shfl_sync(0xffffffffu, dst, from);
                to[u] = (left >> from) & 1 && live ? d : -1;
                if (to[u] >= 0) {
                    x[u] = *row(k, s, p.ckp, p.ckt);
                    y[u] = *row(v, s, p.cvp, p.cvt);
                }
            }
            __syncthreads();                               // all have read what others write
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (to[u] >= 0) {
                    *row(k, to[u], p.ckp, p.ckt) = x[u];
                    *row(v, to[u], p.cvp, p.cvt) = y[u];
                }
        }
    }
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_tree_tables(const int32_t* parents, int64_t parents_stride, int B, int N, const int32_t* n_len, int32_t* mask,
                     int64_t mask_stride_b, int64_t mask_stride_n, int32_t* depth, int64_t depth_stride, void* stream) {
    if (B <= 0 || N <= 0 || parents == nullptr || mask == nullptr || parents_stride < 0) return SAGE_ERR_ARG;
    if (N > kTreeTokens) return SAGE_ERR_UNSUPPORTED;
    const int W = (N + 31) / 32;
    // rows written once
    if ((N > 1 && mask_stride_n < W) || (B > 1 && mask_stride_b < W) || (B > 1 && depth != nullptr && depth_stride < N))
        return SAGE_ERR_ARG;
    TreeParams p{};
    p.parents = parents; p.psb = parents_stride; p.n_len = n_len;
    p.mask = mask; p.msb = mask_stride_b; p.msn = mask_stride_n;
    p.depth = depth; p.dsb = depth_stride;
    p.B = B; p.N = N; p.W = W;
    p.pack = std::max(1, kTreeThreads / 32 / W);
    static bool ready[2][64] = {};
    const dim3 grid((unsigned)ceil_div(B, p.pack), (unsigned)ceil_div(N, kTreeThreads)), block(kTreeThreads);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((N <= kTreeThreads ? launch_pdl(tree_tables_kernel<kTreeThreads>, grid, block, 0, st, 1, false, ready[0], p)
                           : launch_pdl(tree_tables_kernel<kTreeTokens>, grid, block, 0, st, 1, false, ready[1], p)) !=
        cudaSuccess)
        return SAGE_ERR_LAUNCH;
    set_last_launch_count(1);
    return SAGE_OK;
}

int sage_cache_keep(const int32_t* kept, int64_t kept_stride, int B, int K, const int32_t* slots, int64_t slots_stride, int N,
                    const sage_page_cache* cache, void* stream) {
    const int rc = check_page_cache(cache);
    if (rc != SAGE_OK) return rc;
    if (B <= 0 || K <= 0 || N < K || kept == nullptr || slots == nullptr || kept_stride < 0 || slots_stride < 0)
        return SAGE_ERR_ARG;
    KeepParams p{};
    p.status = device_status_ptr();
    if (p.status == nullptr) return SAGE_ERR_LAUNCH;
    p.kept = kept; p.kept_stride = kept_stride; p.slots = slots; p.slots_stride = slots_stride;
    p.ck = static_cast<uint16_t*>(const_cast<void*>(cache->k.ptr));
    p.cv = static_cast<uint16_t*>(const_cast<void*>(cache->v.ptr));
    p.ckp = cache->k.stride_b; p.ckh = cache->k.stride_h; p.ckt = cache->k.stride_n;
    p.cvp = cache->v.stride_b; p.cvh = cache->v.stride_h; p.cvt = cache->v.stride_n;
    p.capacity = (int64_t)cache->num_pages * cache->page_size;
    p.N = N; p.K = K;
    p.chunk_shift = cache->D == 128 ? 4 : 3;
    p.columns = cache->heads << p.chunk_shift;
    p.page = cache->page_size;
    p.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
    static bool ready[2][64] = {};
    const dim3 grid((unsigned)B, (unsigned)ceil_div(p.columns, kKeepColumns));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Four groups of a block share the moves of a call of few blocks and several entries.
    // Such a block holds 256 threads of 104 registers, and two run on an SM at a time:
    //  - up to two blocks an SM, from the seventh entry on, as one group has six moves in
    //    flight (16 heads of 128, 256 blocks, 8 entries: 2.9 us, one group 3.2; 7 entries
    //    2.9 and 2.9; 20: 3.5 and 5.9; 16 requests, 4 heads of 64, up to 91: 5.9 and 16.3);
    //  - up to four, in two rounds, from the eleventh on (336 blocks, 7 entries: 3.5 and
    //    2.9; 10: 3.7 and 3.8; 12: 3.9 and 4.15; 608 blocks, 7: 3.9 and 3.1; 10: 4.3 and
    //    4.3; 12: 4.5 and 4.8; 20: 5.8 and 8.1);
    //  - beyond, one group, whose blocks hide each other's waits (704 blocks, 12 entries:
    //    5.4 and 4.7; 2,048, 20: 19.3 and 16.4; but 920, 20: 9.2 and 10.3).
    const int64_t blocks = (int64_t)grid.x * grid.y;
    const int sms = sm_count();
    const bool one = blocks > 4 * sms || K <= (blocks > 2 * sms ? 10 : 6);
    if ((one ? launch_pdl(cache_keep_kernel<1>, grid, dim3(kKeepColumns), 0, st, 1, false, ready[0], p)
               : launch_pdl(cache_keep_kernel<4>, grid, dim3(kKeepColumns * 4), 0, st, 1, false, ready[1], p)) != cudaSuccess)
        return SAGE_ERR_LAUNCH;
    set_last_launch_count(1);
    return SAGE_OK;
}

}  // extern "C"
