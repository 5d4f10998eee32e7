// sage_tables.cu - the bookkeeping of a page cache on the GPU: page tables and
// slot maps from request lengths, and the append of new keys and values.
#include <algorithm>

#include "sage_gb300.h"
#include "sage_internal.h"
#include "sage_paged.h"

namespace sage {
namespace {

// ---------------------------------------------------------------------------
// Page tables and slots.
//
// Request b holds p(old) = ceil(old / P) pages and needs p(new); it takes the
// pages free[first .. first + need) with first = sum of the needs before it.
// One launch: every block sums the needs in front of its first request itself
// (8 bytes per request, from L2 for all blocks but the first), which costs
// less than a second launch or a wait between blocks.
// ---------------------------------------------------------------------------
struct TableParams {
    const int32_t* old_len;              // or null: 0
    const int32_t* new_len;
    const int32_t* free_pages;
    int32_t* table;
    int32_t* slots;
    int32_t* taken;
    int64_t table_stride, slots_stride;
    int B, W, N, n_free, page, page_shift;
    bool len_quads;                      // the lengths are 16-byte aligned
};

struct Held { int old_len, new_len, old_pages, new_pages; };

__device__ __forceinline__ Held held(const TableParams& p, int o, int n) {
    Held x;
    const int cap = p.W << p.page_shift;                   // at most 2^31 - 1 - page
    x.old_len = min(max(o, 0), cap);
    x.new_len = max(x.old_len, min(max(n, 0), cap));
    x.old_pages = (x.old_len + p.page - 1) >> p.page_shift;
    x.new_pages = (x.new_len + p.page - 1) >> p.page_shift;
    return x;
}
__device__ __forceinline__ Held held(const TableParams& p, int b) {
    return held(p, p.old_len == nullptr ? 0 : p.old_len[b], p.new_len[b]);
}

constexpr int kTableThreads = 256;

// kQuads: rows of the table and of the slots are 16-byte aligned and a multiple
// of 4 long; they leave four entries a store.  A large batch is bound by
// instructions: about 25 an entry one by one, half as many in fours (2,048 rows
// of 1,024 pages and 1,024 slots: 7.8 us one by one, 6.6 in fours).
template <bool kQuads>
__global__ void __launch_bounds__(kTableThreads, 8) page_tables_kernel(const __grid_constant__ TableParams p) {
    __shared__ int red[kTableThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int per = (p.B + gridDim.x - 1) / gridDim.x;
    const int b0 = min((int)blockIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    if (b0 == b1) return;
    Held x = held(p, b0);
    int sum = 0;
    int quads = 0;                                         // requests counted four at a time
    if (p.len_quads) {
        quads = b0 & ~3;
#pragma unroll 2
        for (int b = 4 * (int)threadIdx.x; b < quads; b += 4 * kTableThreads) {
            const int4 n = *reinterpret_cast<const int4*>(p.new_len + b);
            const int4 o = p.old_len == nullptr ? make_int4(0, 0, 0, 0) : *reinterpret_cast<const int4*>(p.old_len + b);
            const int nn[4] = {n.x, n.y, n.z, n.w}, oo[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Held y = held(p, oo[e], nn[e]);
                sum += y.new_pages - y.old_pages;
            }
        }
    }
    for (int b = quads + (int)threadIdx.x; b < b0; b += kTableThreads) {
        const Held y = held(p, b);
        sum += y.new_pages - y.old_pages;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
    __syncthreads();
    int first = 0;
#pragma unroll
    for (int i = 0; i < kTableThreads / 32; ++i) first += red[i];
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        if (b > b0) x = held(p, b);
        int32_t* row = p.table + (int64_t)b * p.table_stride;
        // page of entry j of this request after the call, read where it comes
        // from: other threads are writing the row
        auto entry = [&](int j) -> int {
            if (j < x.old_pages) return row[j];
            const int f = first + (j - x.old_pages);
            return j < x.new_pages && f < p.n_free ? p.free_pages[f] : -1;
        };
        // first slot of a page; -1 for none, or when its slots pass 2^31 - 1
        auto slots_of = [&](int pg) -> int {
            return pg >= 0 && pg <= (INT32_MAX >> p.page_shift) ? pg << p.page_shift : -1;
        };
        int32_t* out = p.slots + (int64_t)b * p.slots_stride;
        const int count = x.new_len - x.old_len;           // slots that name a token
        if constexpr (kQuads) {
            // kept entries of the first four are written back as they are
#pragma unroll 1
            for (int j = (x.old_pages & ~3) + 4 * (int)threadIdx.x; j < p.W; j += 4 * kTableThreads)
                *reinterpret_cast<int4*>(row + j) = make_int4(entry(j), entry(j + 1), entry(j + 2), entry(j + 3));
#pragma unroll 1
            for (int i = 4 * (int)threadIdx.x; i < p.N; i += 4 * kTableThreads) {
                int4 s = make_int4(-1, -1, -1, -1);
                if (i < count) {
                    // four tokens lie in two pages at most
                    const int t = x.old_len + i, a = t >> p.page_shift, z = min(t + 3, x.new_len - 1) >> p.page_shift;
                    const int base = slots_of(entry(a)), next = z == a ? base : slots_of(entry(z));
                    auto slot = [&](int e) -> int {
                        const int from = (t + e) >> p.page_shift == a ? base : next;
                        return i + e < count && from >= 0 ? from + ((t + e) & (p.page - 1)) : -1;
                    };
                    s = make_int4(slot(0), slot(1), slot(2), slot(3));
                }
                *reinterpret_cast<int4*>(out + i) = s;
            }
        } else {
#pragma unroll 2
            for (int j = x.old_pages + (int)threadIdx.x; j < p.W; j += kTableThreads) row[j] = entry(j);
#pragma unroll 2
            for (int i = threadIdx.x; i < p.N; i += kTableThreads) {
                int slot = -1;
                if (i < count) {
                    const int t = x.old_len + i, base = slots_of(entry(t >> p.page_shift));
                    if (base >= 0) slot = base + (t & (p.page - 1));
                }
                out[i] = slot;
            }
        }
        first += x.new_pages - x.old_pages;
    }
    if (b1 == p.B && threadIdx.x == 0) *p.taken = first;
}

// ---------------------------------------------------------------------------
// Append: one warp copies the K and V rows of one token, 16 bytes a lane.
// Reads and writes each row once; HBM bounds it (16 prompts of up to 2,048
// tokens, 16 heads of 128 channels: 38 us, the copy's rate 36).  A lane loads
// four chunks of K and of V before it stores them (one chunk: 41.5 us).  Four
// blocks an SM, whose registers hold them; with six they spill (56 us).
// ---------------------------------------------------------------------------
struct AppendParams {
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* ck;
    uint16_t* cv;
    const int32_t* slots;
    int* status;
    int64_t ksb, ksh, ksn, vsb, vsh, vsn;
    int64_t ckp, ckh, ckt, cvp, cvh, cvt;
    int64_t slots_stride, capacity;
    int64_t tokens;                      // B * N, below 2^31
    int N, heads, chunk_shift;           // chunk_shift: log2 of the 16-byte chunks of a head's row
    int page, page_shift;
};

constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads, 4) cache_append_kernel(const __grid_constant__ AppendParams p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int chunks = p.heads << p.chunk_shift;
    const int64_t t = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const int b = (int)((uint32_t)t / (uint32_t)p.N), i = (int)t - b * p.N;
    const int slot = p.slots[b * p.slots_stride + i];
    if (slot < 0) return;
    if (slot >= p.capacity) {
        if (lane == 0 && atomicCAS(p.status, 0, kErrPage) == 0) p.status[3] = slot >> p.page_shift;
        return;
    }
    const int64_t pg = slot >> p.page_shift;
    const int off = slot & (p.page - 1);
    const uint16_t* k = p.k + b * p.ksb + i * p.ksn;
    const uint16_t* v = p.v + b * p.vsb + i * p.vsn;
    uint16_t* ck = p.ck + pg * p.ckp + off * p.ckt;
    uint16_t* cv = p.cv + pg * p.cvp + off * p.cvt;
    constexpr int kFlight = 4;                             // chunks of a lane whose loads precede their stores
#pragma unroll 1
    for (int c0 = lane; c0 < chunks; c0 += 32 * kFlight) {
        uint4 a[kFlight], d[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int c = c0 + 32 * u, h = c >> p.chunk_shift, x = (c - (h << p.chunk_shift)) * 8;
            if (c < chunks) {
                a[u] = *reinterpret_cast<const uint4*>(k + h * p.ksh + x);
                d[u] = *reinterpret_cast<const uint4*>(v + h * p.vsh + x);
            }
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int c = c0 + 32 * u, h = c >> p.chunk_shift, x = (c - (h << p.chunk_shift)) * 8;
            if (c < chunks) {
                *reinterpret_cast<uint4*>(ck + h * p.ckh + x) = a[u];
                *reinterpret_cast<uint4*>(cv + h * p.cvh + x) = d[u];
            }
        }
    }
}

bool page_size_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

}  // namespace

int check_view(const sage_tensor* t) {
    if (t == nullptr || t->ptr == nullptr) return SAGE_ERR_ARG;
    if (!aligned16(t->ptr) || (t->stride_b % 8) || (t->stride_h % 8) || (t->stride_n % 8) ||
        t->stride_b < 0 || t->stride_h < 0 || t->stride_n < 0)
        return SAGE_ERR_UNSUPPORTED;
    return SAGE_OK;
}

int check_page_cache(const sage_page_cache* c) {
    if (c == nullptr || c->num_pages <= 0 || c->heads <= 0 || c->heads > 65535) return SAGE_ERR_ARG;
    if ((c->D != 64 && c->D != 128) || !page_size_ok(c->page_size)) return SAGE_ERR_UNSUPPORTED;
    if ((int64_t)c->num_pages * c->page_size > INT32_MAX) return SAGE_ERR_UNSUPPORTED;
    for (const sage_tensor* t : {&c->k, &c->v}) {
        const int rc = check_view(t);
        if (rc != SAGE_OK) return rc;
        // rows apart (no broadcast axis), and byte strides that a tensor map holds
        if (t->stride_n < c->D || (c->heads > 1 && t->stride_h < c->D) || (c->num_pages > 1 && t->stride_b < c->D))
            return SAGE_ERR_UNSUPPORTED;
        for (int64_t s : {t->stride_b, t->stride_h, t->stride_n})
            if (s >= (int64_t(1) << 38)) return SAGE_ERR_UNSUPPORTED;
    }
    return SAGE_OK;
}

}  // namespace sage

using namespace sage;

extern "C" {

int sage_page_tables(const int32_t* old_len, const int32_t* new_len, int B, int page_size,
                     const int32_t* free_pages, int n_free, int32_t* table, int64_t table_stride, int table_width,
                     int32_t* slots, int64_t slots_stride, int n_slots, int32_t* taken, void* stream) {
    if (B <= 0 || new_len == nullptr || taken == nullptr || table == nullptr || table_width <= 0) return SAGE_ERR_ARG;
    if (n_free < 0 || (n_free > 0 && free_pages == nullptr) || n_slots < 0 || (n_slots > 0 && slots == nullptr))
        return SAGE_ERR_ARG;
    if ((B > 1 && table_stride < table_width) || (B > 1 && n_slots > 0 && slots_stride < n_slots)) return SAGE_ERR_ARG;
    if (!page_size_ok(page_size)) return SAGE_ERR_UNSUPPORTED;
    // lengths and the count of pages taken stay in int
    if ((int64_t)table_width * page_size > INT32_MAX - page_size || (int64_t)B * table_width > INT32_MAX)
        return SAGE_ERR_UNSUPPORTED;
    TableParams p{};
    p.old_len = old_len; p.new_len = new_len; p.free_pages = free_pages; p.n_free = n_free;
    p.table = table; p.table_stride = table_stride; p.W = table_width;
    p.slots = slots; p.slots_stride = slots_stride; p.N = n_slots;
    p.taken = taken; p.B = B; p.page = page_size;
    p.page_shift = 31 - __builtin_clz((unsigned)page_size);
    p.len_quads = aligned16(new_len) && (old_len == nullptr || aligned16(old_len));
    const bool quads = aligned16(table) && table_stride % 4 == 0 && table_width % 4 == 0 &&
                       (n_slots == 0 || (aligned16(slots) && slots_stride % 4 == 0 && n_slots % 4 == 0));
    static bool ready[2][64] = {};
    const dim3 grid((unsigned)std::min(B, 152 * 8)), block(kTableThreads);     // one wave: eight blocks an SM
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((quads ? launch_pdl(page_tables_kernel<true>, grid, block, 0, s, 1, false, ready[1], p)
               : launch_pdl(page_tables_kernel<false>, grid, block, 0, s, 1, false, ready[0], p)) != cudaSuccess)
        return SAGE_ERR_LAUNCH;
    set_last_launch_count(1);
    return SAGE_OK;
}

int sage_cache_append(const sage_tensor* k, const sage_tensor* v, int B, int N, const int32_t* slots,
                      int64_t slots_stride, const sage_page_cache* cache, void* stream) {
    int rc = check_page_cache(cache);
    if (rc != SAGE_OK) return rc;
    if (B <= 0 || N <= 0 || slots == nullptr || slots_stride < 0) return SAGE_ERR_ARG;
    if ((int64_t)B * N > INT32_MAX) return SAGE_ERR_UNSUPPORTED;
    if ((rc = check_view(k)) != SAGE_OK || (rc = check_view(v)) != SAGE_OK) return rc;
    AppendParams p{};
    p.status = device_status_ptr();
    if (p.status == nullptr) return SAGE_ERR_LAUNCH;
    p.k = static_cast<const uint16_t*>(k->ptr);
    p.v = static_cast<const uint16_t*>(v->ptr);
    p.ck = static_cast<uint16_t*>(const_cast<void*>(cache->k.ptr));
    p.cv = static_cast<uint16_t*>(const_cast<void*>(cache->v.ptr));
    p.slots = slots; p.slots_stride = slots_stride;
    p.ksb = k->stride_b; p.ksh = k->stride_h; p.ksn = k->stride_n;
    p.vsb = v->stride_b; p.vsh = v->stride_h; p.vsn = v->stride_n;
    p.ckp = cache->k.stride_b; p.ckh = cache->k.stride_h; p.ckt = cache->k.stride_n;
    p.cvp = cache->v.stride_b; p.cvh = cache->v.stride_h; p.cvt = cache->v.stride_n;
    p.capacity = (int64_t)cache->num_pages * cache->page_size;
    p.tokens = (int64_t)B * N; p.N = N; p.heads = cache->heads;
    p.chunk_shift = cache->D == 128 ? 4 : 3;
    p.page = cache->page_size;
    p.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
    const int64_t grid = ceil_div(p.tokens, kAppendThreads / 32);
    static bool ready[64] = {};
    if (launch_pdl(cache_append_kernel, dim3((unsigned)grid), dim3(kAppendThreads), 0, static_cast<cudaStream_t>(stream), 1, false,
                   ready, p) != cudaSuccess)
        return SAGE_ERR_LAUNCH;
    set_last_launch_count(1);
    return SAGE_OK;
}

}  // extern "C"
