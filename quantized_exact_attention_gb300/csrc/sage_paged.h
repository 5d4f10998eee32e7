// sage_paged.h - parameter blocks of the paged serving kernels, shared by
// their translation units (host and device).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "sage_gb300.h"
#include "sage_internal.h"

namespace sage {

constexpr int kErrPage = -7;             // SAGE_ERR_PAGE as the kernels record it
constexpr int kMaxRowWorkers = 1280;     // warps of the few-rows kernel that take work (8 per SM, 160 SMs at most)
constexpr int kMaxTileWorkers = 160;     // CTAs of the many-rows kernel with two row groups (1 per SM); with one: twice that

// Division by a constant the host knows: (umulhi(n, m) + n) >> s = n / d for
// 0 <= n < 2^31, with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1
// (Granlund and Montgomery's round-up reciprocal).
struct FastDiv {
    uint32_t m, s;
};
inline FastDiv make_fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    return FastDiv{(uint32_t)(((((uint64_t(1) << s) - d) << 32) / d) + 1), s};
}

// An item whose tiles several workers share, named by the second of them.
struct alignas(16) PagedCut {
    int b, h, rt, n;                     // request (-1: none), key head, row set, query tokens
    int parts;                           // workers that share it
    int pad[3];
};

struct PagedParams {
    const uint16_t* q;                   // BF16 bit patterns
    uint16_t* o;
    const uint16_t* k;                   // page caches [page][head][token][channel] by strides
    const uint16_t* v;
    int64_t qsb, qsh, qsn, osb, osh, osn;            // element strides
    int64_t ksp, ksh, kst, vsp, vsh, vst;            // page, head, token strides
    const int32_t* q_len;                // device [B] or null
    const int32_t* kv_len;               // device [B] or null: own tokens of each request
    const int32_t* prefix_len;           // device [1] or null
    const int32_t* table;                // device [B][table_stride], W entries used
    const int32_t* ptable;               // device [Wp]
    int64_t table_stride;
    int B, H, Hkv, G, Nq;                // G = H / Hkv query heads to a key head
    int W, Wp;                           // table widths in pages (Wp = 0: no prefix)
    int num_pages, page, page_shift;     // tokens per page: a power of two
    int causal;
    float sc;                            // sm_scale * log2(e)
    int* status;
    // schedule (see sage_paged_sched.cuh)
    int rt;                              // row sets of a request
    int pre_rt;                          // row sets of all requests against the prefix (0: a list of own keys)
    int tok;                             // tiles kernel: tokens of a 128-row group
    FastDiv by_G, by_rt;                 // G, rt
    int join;                            // 1: a request's key sequence is the prefix followed by its own keys
    int workers;                         // workers the list is shared among
    int fault_mode;                      // test hook: 0 = none
    int split;                           // few-rows kernel, whole items: CTAs of a cluster
    int whole;                           // many-rows kernel: a CTA takes an item
    int beside;                          // runs beside the kernel before it, which it does not depend on
    // workspace
    float* part_o;                       // [slot][part_m][D]
    float2* part_ml;                     // [slot][part_m] running maximum (log2 domain) and sum
    int part_m;                          // rows of a slot
    PagedCut* cuts;                      // [workers] items that a worker boundary cuts (null: not wanted)
    int32_t* start;                      // [B rt + 1] list position of each (request, row set); last: the length
    // the shared prefix's items, and the list they are in for the join
    float* pre_o;                        // [slot][pre_m][D]
    float2* pre_ml;
    int pre_items_rt, pre_m, pre_workers;            // row sets (0: no such items), rows of an item, workers
    int pre_tok, pre_unit;               // requests of a 128-row group, rows of a request
    FastDiv by_pre_unit;
};

// The many-rows kernel (sage_paged_tiles.cu): workers = CTAs, groups: row groups
// of 128 of an item (1 or 2).  Writes whole rows unless the list holds shared
// prefix items; then every result is partial.  tq: q in boxes of `tok` tokens,
// tqp: of `pre_tok` requests (either may stand for one that no item uses).
cudaError_t launch_paged_tiles(const PagedParams& p, int D, int groups, const CUtensorMap& tq, const CUtensorMap& tqp,
                               const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);

// Tensor map over one tensor of a page cache, box: one page of one head, 64 channels (sage_api.cu).
int encode_pages(CUtensorMap* m, const sage_tensor& t, int D, int page, int heads, int pages);
// Tensor map over q [B, H, Nq, D] as (channel, head, token, request), box: 64
// channels of `heads` heads, `tokens` tokens and `requests` requests.
int encode_rows(CUtensorMap* m, const sage_tensor& t, int D, int H, int Nq, int B, int heads, int tokens, int requests);
// The fault the next launch has to make (test hook), taken once (sage_api.cu).
int take_fault_mode();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Checks of a tensor's and of a page cache's description that need no GPU (sage_tables.cu).
int check_view(const sage_tensor* t);
int check_page_cache(const sage_page_cache* c);

#ifdef __CUDACC__
// Programmatic dependent launch: a kernel may start once every CTA of the
// kernel before it in the stream has called pdl_trigger (or ended), which hides
// its launch and its prologue; pdl_wait returns when that kernel is complete
// and its writes are visible.  Every CTA of every kernel here calls pdl_wait
// before it ends, so a kernel that is complete has nothing unfinished before
// it.  The first kernel of an attention call waits before it triggers: what
// follows it within the call may read the caller's tensors at once.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Loads of what an earlier kernel of the stream may have written (lengths,
// tables, slots, new rows, partial results).  This kernel's life begins before
// that one ends, so they are not __ldg's, which is for data that nothing writes
// while the kernel lives; and the compiler may move __ldg and __ldcg above
// pdl_wait.  A plain load stays behind it, and sees all that was waited for.
// A kernel may read before its own pdl_wait what was complete when the kernel
// before it, which waited, let it start.  Such values are in L2, but nothing has
// emptied this SM's L1 since: either a fence does first, or the load goes past it.
__device__ __forceinline__ void fence_before_early_loads() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }
__device__ __forceinline__ int ld_gpu(const int32_t* a) {
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");
    return v;
}

// Launch a kernel this way.  The kernels of an attention call ask for the same
// split of an SM's memory (`max_shared`, set once per device): an SM drains
// before it changes the split (a short decode call: 10.4 us, with the same
// split 9.0 us).  The append moves its rows through L1 and keeps the default
// (2 x 122 MB: 37.9 us; with little L1 46.3).
template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                       bool max_shared, bool (&ready)[64], const A&... args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        if (max_shared && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                    (int)cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
        if (smem > 0 && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
            return e;
        ready[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}
#endif

}  // namespace sage
