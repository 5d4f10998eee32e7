// sage_paged.cu - attention over a page cache, for a batch that may share a
// prefix: the kernel for few query rows, the kernel that joins partial
// results, and the C entry points.
//
// Row (b, h, i) sees the prefix's keys and its request's own keys j < kv_len[b]
// (causal: j <= i + kv_len[b] - q_len[b]):
//     o = sum_j softmax_j(sm_scale * q.k_j) v_j        (no key: 0)
// The softmax runs online: per key tile the running maximum m, the sum
// l = sum 2^(s - m) and O = sum 2^(s - m) v are updated in FP32 (s in the log2
// domain).  Results over disjoint key sets join exactly the same way:
//     M = max m_p,  o = (sum_p 2^(m_p - M) O_p) / (sum_p 2^(m_p - M) l_p),
// which is what lets one request's keys be split among workers and the
// prefix be read once for the rows of all requests.
#include <algorithm>
#include <cmath>

#include "sage_gb300.h"
#include "sage_internal.h"
#include "sage_paged.h"
#include "sage_paged_sched.cuh"
#include "sage_ptx.cuh"
#include "sage_quant.cuh"

namespace sage {
namespace {

// ---------------------------------------------------------------------------
// Few rows: one warp is one worker.
//
// Reading the keys and values bounds this form (per key 4*D bytes, and only
// 4*D operations for each of a few rows), so the work of a warp is a stream
// of 16-key steps through its own ring of shared-memory stages, filled by
// 16-byte asynchronous copies; no barrier joins the warps of a CTA.
// S^T = K Q^T and O^T = V^T P^T, i.e. the keys (then the channels) are the
// 16 rows of the matrix instruction and the query rows its 8 columns, so 8
// query rows waste nothing, and the rescale factor of a query row multiplies
// whole accumulator columns.  P is rounded to BF16 (relative error at most 2^-8) for
// the second product, as its other operand V is BF16; l sums it unrounded.
// A step never crosses a page: pages hold a multiple of 16 tokens.
// Measured, a call with its join: 64 ragged requests of up to 8,192 keys (1,077
// MB read) in 166 to 171 us, 0.93 to 0.96 of the copy rate; one of 131,072 keys
// (537 MB) in 89 to 91 us, 0.87 to 0.89.
// Beside the prefix's kernel it reads lengths, pages and rows before its own
// wait, behind a fence (128 requests behind 16,333 shared keys: 88 to 89 us a
// call; with relaxed loads, which go past L1, in its place 92).
// kWhole: for short sequences, bound by latency, a cluster of `split` CTAs
// takes an item, shares its steps among its warps and joins them through
// shared memory, so the call is one kernel (8 key heads, 60 keys: 3.9 us
// against 6.6 with the join behind it; 777 keys: 6.7 against 7.4).
// ---------------------------------------------------------------------------
constexpr int kRowWarps = 4;             // warps of a CTA
constexpr int kStep = 16;                // keys of a step

template <int D>
struct RowsShape {
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kChunks = D / 8;                          // 16-byte chunks of a row
    static constexpr uint32_t kTile = kStep * D * 2;               // K (or V) bytes of a stage
    static constexpr uint32_t kStage = 2 * kTile;
    static constexpr uint32_t kSmem = kRowWarps * kStages * kStage;
};

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void record_page(const PagedParams& p, int page) {
    if (atomicCAS(p.status, 0, kErrPage) == 0) p.status[3] = page;
}

// A step as the loading side leaves it for the computing side.
struct StepNote {
    int b, h, rt, item;                  // of its item
    int n, len;                          // the request's query tokens and own keys
    int key0, nkeys;
    int own, first;                      // own keys; first step of its item in this warp
};

template <int D, int NR, bool kWhole>
__global__ void __launch_bounds__(kRowWarps * 32, 2) paged_rows_kernel(const __grid_constant__ PagedParams p) {
    using Sh = RowsShape<D>;
    constexpr int M = 8 * NR, S = Sh::kStages;
    constexpr int kRowsPerPass = 32 / Sh::kChunks;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int2 found[kRowWarps];
    __shared__ int warp_sums[kRowWarps];
    __shared__ StepNote notes[kRowWarps][S];
    __shared__ float2 part_ml[kRowWarps][M];
    constexpr int kPartRow = D + 4;                       // floats; rows two apart lie in other banks
    static_assert(M * kPartRow * 4 <= S * Sh::kStage && (S * Sh::kStage) % 16 == 0);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!kWhole && p.beside) fence_before_early_loads();
    else pdl_wait();
    pdl_trigger();
    const PagedSched<M, kStep, false> sched(p);
    int worker, t1;                                       // this worker, the end of its run of places
    int parts = 0;                                        // kWhole: workers that share the item
    PagedPlace at{};
    if constexpr (kWhole) {
        const int all = (int)blockIdx.x / p.split;        // a cluster takes an item
        worker = ((int)blockIdx.x - all * p.split) * kRowWarps + warp;
        const int pair = all / p.Hkv;
        at.h = all - pair * p.Hkv;
        at.b = pair / p.rt;
        at.rt = pair - at.b * p.rt;
        at.n = sched.q_rows(at.b);
        at.len = sched.own_keys(at.b);
        at.ntiles = sched.item_tiles(at.n, at.len, at.rt);
        const int workers = p.split * kRowWarps, per = max(1, (at.ntiles + workers - 1) / workers);
        parts = (at.ntiles + per - 1) / per;
        at.tile = at.pos = min(worker * per, at.ntiles);
        t1 = min(at.pos + per, at.ntiles);
    } else {
        // workers next to each other in the list sit on different SMs: a CTA's
        // warps are a grid apart, so a short list still uses every SM
        worker = warp * gridDim.x + blockIdx.x;
        const int total = paged_scan<M, kStep, false, kRowWarps * 32, kRowWarps>(sched, blockIdx.x, gridDim.x, found,
                                                                                 warp_sums, blockIdx.x == 0);
        const int per = sched.share(total, p.workers, p.B * p.rt * p.Hkv), t0 = min(worker * per, total);
        t1 = min(t0 + per, total);
        at.pos = t1;
        if (t0 < t1) at = paged_place(sched, found[warp], t0);
        if (at.pos >= t1) {
            pdl_wait();
            return;
        }
    }
    const uint32_t ring = smem_u32(smem) + warp * S * Sh::kStage;
    int issued = 0;                                       // steps whose copies were issued
    bool first = true;
    PagedSpan span{};
    int page = 0;
    // Read the page number of the next step (one step before its copies, so
    // that the table's latency lies behind a step of computing).
    auto fetch = [&]() {
        span = paged_span(sched, at.b, at.len, at.tile);
        const int j = span.key0 >> p.page_shift;
        page = span.own ? p.table[(int64_t)at.b * p.table_stride + j] : p.ptable[j];
    };
    auto issue = [&](int stage) {
        const bool ok = (unsigned)page < (unsigned)p.num_pages;
        if (!ok && lane == 0) record_page(p, page);
        const int nk = ok ? span.nkeys : 0;               // rows of a page outside the cache read as zero
        const int64_t pg = ok ? page : 0;
        const int off = span.key0 & (p.page - 1);
        const int r0 = lane / Sh::kChunks, c = lane % Sh::kChunks;
        const uint16_t* kp = p.k + pg * p.ksp + at.h * p.ksh + (int64_t)(off + r0) * p.kst + c * 8;
        const uint16_t* vp = p.v + pg * p.vsp + at.h * p.vsh + (int64_t)(off + r0) * p.vst + c * 8;
        const uint32_t base = ring + stage * Sh::kStage;
#pragma unroll
        for (int i = 0; i < kStep / kRowsPerPass; ++i) {
            const int r = r0 + i * kRowsPerPass;
            const uint32_t d = base + r * (D * 2) + ((c ^ (r & 7)) << 4);
            const bool in = r < nk;
            cp_async16(d, in ? kp + (int64_t)i * kRowsPerPass * p.kst : p.k, in ? 16u : 0u);
            cp_async16(d + Sh::kTile, in ? vp + (int64_t)i * kRowsPerPass * p.vst : p.v, in ? 16u : 0u);
        }
        if (lane == 0) {
            StepNote& nt = notes[warp][stage];
            nt.b = at.b; nt.h = at.h; nt.rt = at.rt; nt.item = at.item;
            nt.n = at.n; nt.len = at.len;
            nt.key0 = span.key0; nt.nkeys = span.nkeys;
            nt.own = span.own; nt.first = first;
        }
        ++issued;
        if constexpr (kWhole) {
            ++at.pos;
            ++at.tile;
            first = false;
        } else {
            const int item = at.item;
            paged_next(sched, at);
            first = at.item != item;
        }
        if (at.pos < t1) fetch();
    };

    if (at.pos < t1) fetch();

    uint32_t qf[NR][D / 16][2];                           // Q^T fragments
    float o[NR][D / 16][4];                               // O^T: channels x query rows
    float m[NR][2], l[NR][2];                             // of the two query rows this lane's columns are
    int lim[NR][2];                                       // own keys each of them sees
    int item = -1, ib = 0, ih = 0, irt = 0, tokens = 0;   // the item these belong to, its request's query tokens

    // Leave the item's partial result.
    auto leave = [&]() {
        const int64_t slot = (int64_t)worker + item;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float s = l[nr][e];
                s += __shfl_xor_sync(0xffffffffu, s, 4);
                s += __shfl_xor_sync(0xffffffffu, s, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 16);
                const int r = nr * 8 + (lane & 3) * 2 + e;
                int b, i, hq;
                float* dst;
                if constexpr (kWhole) {                   // in place of the ring
                    if (lane < 4) part_ml[warp][r] = make_float2(m[nr][e], s);
                    dst = reinterpret_cast<float*>(smem + warp * S * Sh::kStage) + r * kPartRow + (lane >> 2);
                } else {
                    if (!paged_row(sched, ib, ih, irt, tokens, r, b, i, hq)) continue;
                    if (lane < 4) p.part_ml[slot * M + r] = make_float2(m[nr][e], s);
                    dst = p.part_o + (slot * M + r) * D + (lane >> 2);
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    dst[j * 16] = o[nr][j][e];
                    dst[j * 16 + 8] = o[nr][j][2 + e];
                }
            }
        }
    };
    auto enter = [&](const StepNote& nt) {
        item = nt.item; ib = nt.b; ih = nt.h; irt = nt.rt;
        const int n = nt.n, len = nt.len;
        tokens = n;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            int b, i, hq;
            const bool in = paged_row(sched, ib, ih, irt, n, nr * 8 + (lane >> 2), b, i, hq);
            const uint16_t* qp = p.q + (in ? b * p.qsb + hq * p.qsh + i * p.qsn : 0) + (lane & 3) * 2;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                qf[nr][j][0] = in ? *reinterpret_cast<const uint32_t*>(qp + j * 16) : 0u;
                qf[nr][j][1] = in ? *reinterpret_cast<const uint32_t*>(qp + j * 16 + 8) : 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nr][j][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nr][e] = -INFINITY;
                l[nr][e] = 0.f;
                lim[nr][e] = len;
                if (p.causal) {
                    const int rr = irt * M + nr * 8 + (lane & 3) * 2 + e;
                    lim[nr][e] = min(len, len - n + fast_div(rr, p.by_G) + 1);
                }
            }
        }
    };

    // The ring is filled by the same loop (one copy of its code): S - 1 steps
    // that only load.
    int stage = 0, fill = 0;                              // stages to compute from and to load into
#pragma unroll 1
    for (int it = 1 - S; it < 0 || it < issued; ++it) {
        cp_async_wait<S - 2>();
        __syncwarp();
        const StepNote nt = notes[warp][stage];
        if (at.pos < t1) issue(fill);                        // its stage was read in the step before
        fill = fill + 1 == S ? 0 : fill + 1;
        cp_async_commit();
        if (it < 0) continue;
        if (nt.first) {
            if (it > 0) leave();
            enter(nt);
        }
        const uint32_t kb = ring + stage * Sh::kStage, vb = kb + Sh::kTile;
        stage = stage + 1 == S ? 0 : stage + 1;
        float sacc[NR][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 4; ++e) sacc[nr][e] = 0.f;
        {
            const int r = lane & 15;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t a[4];
                ldsm_x4(a, kb + r * (D * 2) + (((2 * j + (lane >> 4)) ^ (r & 7)) << 4));
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) mma_bf16(sacc[nr], a, qf[nr][j][0], qf[nr][j][1]);
            }
        }
        uint32_t pf[NR][2];
        const int k0 = nt.key0 + (lane >> 2);             // this lane's keys: k0 and k0 + 8
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int end = nt.own ? min(lim[nr][e], nt.key0 + nt.nkeys) : nt.key0 + nt.nkeys;
                if (k0 >= end) sacc[nr][e] = -INFINITY;
                if (k0 + 8 >= end) sacc[nr][2 + e] = -INFINITY;
                float mx = fmaxf(sacc[nr][e], sacc[nr][2 + e]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[nr][e], mx * p.sc);
                const float ms = mn == -INFINITY ? 0.f : mn;      // no visible key yet: every weight is 0
                f[e] = ex2_approx(m[nr][e] - ms);
                m[nr][e] = mn;
                sacc[nr][e] = ex2_approx(fmaf(sacc[nr][e], p.sc, -ms));
                sacc[nr][2 + e] = ex2_approx(fmaf(sacc[nr][2 + e], p.sc, -ms));
                l[nr][e] = l[nr][e] * f[e] + (sacc[nr][e] + sacc[nr][2 + e]);
            }
            pf[nr][0] = transpose8x8(pack_bf16(sacc[nr][0], sacc[nr][1]));
            pf[nr][1] = transpose8x8(pack_bf16(sacc[nr][2], sacc[nr][3]));
            if (!__all_sync(0xffffffffu, f[0] == 1.f && f[1] == 1.f)) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    o[nr][j][0] *= f[0]; o[nr][j][1] *= f[1];
                    o[nr][j][2] *= f[0]; o[nr][j][3] *= f[1];
                }
            }
        }
        {
            const int r = (lane & 7) + ((lane >> 4) << 3), hc = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t a[4];
                ldsm_x4_t(a, vb + r * (D * 2) + (((2 * j + hc) ^ (r & 7)) << 4));
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) mma_bf16(o[nr][j], a, pf[nr][0], pf[nr][1]);
            }
        }
    }
    cp_async_wait<0>();
    if constexpr (kWhole) {
        __syncwarp();
        if (issued > 0) leave();
        __syncwarp();
        cluster_sync_all();
        // Join the workers' parts: a thread takes four channels of a row at a time.
        const int rank = (int)blockIdx.x % p.split;
        for (int v = rank * (int)blockDim.x + (int)threadIdx.x; v < M * D / 4; v += p.split * (int)blockDim.x) {
            const int r = v / (D / 4), c = (v - r * (D / 4)) * 4;
            int b, i, hq;
            if (!paged_row(sched, at.b, at.h, at.rt, at.n, r, b, i, hq)) continue;
            const uint32_t ml0 = smem_u32(&part_ml[0][r]), o0 = smem_u32(smem) + (uint32_t)(r * kPartRow + c) * 4;
            float mx = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = 0; w < parts; ++w) {
                const uint32_t cta = (uint32_t)w / kRowWarps, in = (uint32_t)w % kRowWarps;
                const float2 ml = ld_cluster2(mapa_rank(ml0 + in * (uint32_t)sizeof(part_ml[0]), cta));
                const float4 x = ld_cluster4(mapa_rank(o0 + in * S * Sh::kStage, cta));
                const float mn = fmaxf(mx, ml.x), ms = mn == -INFINITY ? 0.f : mn;
                const float fa = ex2_approx(mx - ms), fb = ex2_approx(ml.x - ms);
                l = l * fa + ml.y * fb;
                acc.x = acc.x * fa + x.x * fb;
                acc.y = acc.y * fa + x.y * fb;
                acc.z = acc.z * fa + x.z * fb;
                acc.w = acc.w * fa + x.w * fb;
                mx = mn;
            }
            // as in the join kernel: l is 0 exactly when the row saw no key
            const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
            uint16_t* dst = p.o + b * p.osb + hq * p.osh + (int64_t)i * p.osn + c;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        }
        __syncwarp();
        cluster_sync_all();                                // the parts stay until all have read them
    } else {
        leave();
        pdl_wait();                      // the prefix's kernel, where one runs beside this one, is through too
    }
}

// ---------------------------------------------------------------------------
// Join the partial results of each output row.  WPR warps share a row.  Bound
// by latency: the parts' loads, four in flight, behind the lookup of where they
// lie (3.3 us after a short decode's rows).
// ---------------------------------------------------------------------------
struct RowParts {
    int64_t slot0;                       // slots slot0, slot0 + 1, ... (one per worker in order)
    int n;
};

// Parts of the item whose `nt` tiles lie from place `start` on.
__device__ __forceinline__ RowParts parts_of(int start, int nt, int per, int item) {
    RowParts r{0, 0};
    if (nt > 0) {
        const int w0 = start / per, w1 = (start + nt - 1) / per;
        r.slot0 = (int64_t)w0 + item;
        r.n = w1 - w0 + 1;
    }
    return r;
}

template <int D, int M, int TK, int WPR>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p) {
    constexpr int V = D / 32;                              // channels of a lane
    constexpr int kFlight = 4;                             // parts whose loads are in flight together
    __shared__ float red_o[8][D];
    __shared__ float2 red_ml[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = (int)blockIdx.x * (8 / WPR) + warp / WPR, sub = warp % WPR;
    const int b = blockIdx.y;
    constexpr bool kTiles = TK == 128;                     // a list of the many-rows kernel, the prefix's items in it
    const PagedSched<M, TK, kTiles> s(p, true);
    const int hq = row / p.Nq, i = row - hq * p.Nq;
    const int n = s.q_rows(b), len = s.own_keys(b);
    const bool live = hq < p.H && i < n;
    const int h = fast_div(hq, p.by_G), r = i * p.G + (hq - h * p.G);
    const int rt = kTiles ? 0 : r / M;  // tiles: one group holds a request's rows
    pdl_trigger();
    pdl_wait();                                            // the parts are written
    float acc[V], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    if (live) {
        const int per = s.share(p.start[p.B * p.rt], p.workers, p.B * p.rt * p.Hkv);
        const int nt = s.item_tiles(n, len, rt), pair = b * p.rt + rt;
        const RowParts own = parts_of(p.start[pair] + h * s.places(nt) + s.kItemCost, nt, per, pair * p.Hkv + h);
        const int64_t own_q = own.slot0 * p.part_m + (r - rt * M);
        RowParts pre{0, 0};
        int64_t pre_q = 0;
        if (p.pre_items_rt > 0) {
            // the row set of the prefix that holds this row, and its place there
            using Tiles = PagedSched<128, 128, true>;
            const int pt = (s.lp + 127) / 128, group = b / p.pre_tok;
            const int set = group * 128 / p.pre_m, place = group * 128 - set * p.pre_m + (b - group * p.pre_tok) * p.Nq * p.G + r;
            const int it = set * p.Hkv + h;
            // ... in the same list, or in one of its own
            const int pre_per = kTiles ? per
                                : Tiles::share(p.Hkv * p.pre_items_rt * Tiles::places(pt), p.pre_workers, 0);
            pre = parts_of(it * Tiles::places(pt) + Tiles::kItemCost, pt, pre_per, it);
            pre_q = pre.slot0 * p.pre_m + place;
        }
        const int parts = own.n + pre.n;
#pragma unroll 1
        for (int x0 = sub; x0 < parts; x0 += kFlight * WPR) {
            float2 ml[kFlight];
            float w[kFlight][V];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const int x = x0 + k * WPR;
                ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int v = 0; v < V; ++v) w[k][v] = 0.f;
                if (x < parts) {
                    const bool from_pre = x < pre.n;
                    const int64_t q = from_pre ? pre_q + (int64_t)x * p.pre_m : own_q + (int64_t)(x - pre.n) * p.part_m;
                    ml[k] = (from_pre ? p.pre_ml : p.part_ml)[q];
                    const float* po = (from_pre ? p.pre_o : p.part_o) + q * D + lane * V;
                    if (V == 4) {
                        const float4 y = *reinterpret_cast<const float4*>(po);
                        w[k][0] = y.x; w[k][1] = y.y; w[k][V - 2] = y.z; w[k][V - 1] = y.w;
                    } else {
                        const float2 y = *reinterpret_cast<const float2*>(po);
                        w[k][0] = y.x; w[k][1] = y.y;
                    }
                }
            }
            float mn = m;
#pragma unroll
            for (int k = 0; k < kFlight; ++k) mn = fmaxf(mn, ml[k].x);
            const float ms = mn == -INFINITY ? 0.f : mn;
            const float fa = ex2_approx(m - ms);
            l *= fa;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= fa;
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const float fb = ex2_approx(ml[k].x - ms);
                l += ml[k].y * fb;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] += w[k][v] * fb;
            }
            m = mn;
        }
    }
    if (WPR > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) red_o[warp][lane * V + v] = acc[v];
        if (lane == 0) red_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (sub != 0) return;
        float mn = m;
#pragma unroll
        for (int x = 1; x < WPR; ++x) mn = fmaxf(mn, red_ml[warp + x].x);
        const float ms = mn == -INFINITY ? 0.f : mn;
        l = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll
        for (int x = 0; x < WPR; ++x) {
            const float fb = ex2_approx(red_ml[warp + x].x - ms);
            l += red_ml[warp + x].y * fb;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += red_o[warp + x][lane * V + v] * fb;
        }
    }
    if (!live) return;
    // l is 0 exactly when the row saw no key (its largest weight is 1); a NaN
    // in l stays in the output
    const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    uint32_t out[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; ++v) out[v] = pack_bf16(acc[2 * v] * inv, acc[2 * v + 1] * inv);
    uint16_t* dst = p.o + b * p.osb + hq * p.osh + (int64_t)i * p.osn + lane * V;
    if (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[V / 2 - 1]);
    else *reinterpret_cast<uint32_t*>(dst) = out[0];
}

// ---------------------------------------------------------------------------
// Host side: which kernel reads which keys for which rows.
//
// A request brings rows = Nq * G query rows to a key head.
//  - rows > 16: the many-rows kernel, each request's keys behind the prefix
//    (one list; the prefix is read again for every request, mostly from L2).
//    Rows that fill a quarter of its 128 waste tensor work that reading the
//    keys hides: 16 requests of 24 rows and up to 4,000 keys take 37 us, in a
//    32-row form of the few-rows kernel 62; 8 of 32 rows and up to 16,000, 57
//    and 94.  (More than 128 query heads to a key head leave no whole token in
//    a group: these, which no model is known to have, stay with the few-rows
//    kernel.)
//    A CTA takes an item whole, with no list and no join behind it, while that
//    leaves few of them idle: items of up to T tiles times groups (by the table
//    widths), half of that on average, for r items a CTA, waste T (1 - r / 2) of
//    a CTA's time, which may be 12; later items start as CTAs end, the longest
//    (of a causal mask) first.  4 requests of 32 tokens, 8 key heads, 500 keys:
//    14.0 us from the list, 9.8 so; 16 heads of 2,048 tokens, two prompts, D =
//    64, T = 32, r = 1.7: 42.6 and 33.4; on the other side 8 heads of 4,096
//    tokens, T = 64, r = 0.8: 50.5 and 63.3; 128 items of 24 rows and up to
//    4,000 keys, T = 32: 36.5 and 53.5; 16 x 16 heads of 1,024 tokens, r = 6.7:
//    112 and 124, the start of every CTA.
//    Requests of more than one group take two to an item, but one where whole
//    items then run all at a time or have up to four tiles: 8 heads of 256 tokens
//    11.6 and 9.3 us, 20 x 16 of 200 25.0 and 19.9; 32 of 2,048 tokens, which do
//    not, 45.3 and 48.5.
//    Up to 64 rows, of which two requests or more fill a group, the prefix may
//    have items of its own in front of the requests', each for the rows of
//    several requests.  That saves tiles and costs a join of all rows, about
//    as much as 12 MB of tiles and 6 KB for each row (32 requests of 20 rows, 8
//    key heads of 128 channels, 8,192 shared keys: 51 us against 125; 4 key
//    heads of 64, 4,099 keys: 22 against 30; on the other side 200 requests of
//    21 rows, 512 shared keys: 34 against 32.5; 16 of 64 rows, 2 key heads,
//    4,096: 20.5 against 17.5).
//  - rows <= 16: the few-rows kernel, each request's keys behind the prefix
//    while reading the prefix again for every request costs less than a list
//    of its own, which the many-rows kernel then reads once for all rows: 64
//    requests, 8 key heads, 512 shared keys (134 MB read again) take 35 us so
//    and 43 with a list, 1,024 keys (268 MB) 44 and 43, 2,048 keys 64 and 44; 16
//    requests, 4,096 keys (268 MB) 32 and 23.
//    Without a list of its own: up to four items an SM take a cluster each when
//    the table widths bound a warp's share to 12 steps, a cluster of 2, 4 or 8
//    CTAs counted as 2, 3 or 4 steps more.  A cluster does not even out the
//    lengths: 38 requests, 8 key heads, one request of n keys and 37 of 30 take
//    5.9 us for n = 250 and 8.9 for 500 so, 8.3 both from a list; at 1,000 (16
//    steps) 14.4 and 9.1, though with 1,000 keys each 27.8 and 32.3.  Eight
//    items an SM of 30 keys: 13.3 us, from a list 9.5; four 7.4 and 8.3.
// ---------------------------------------------------------------------------
constexpr int kFewRows = 16;
constexpr int64_t kReadAgain = int64_t(128) << 20;        // bytes of prefix read again that cost as much as its list
constexpr int kWholeSteps = 12, kWholeItems = 4;          // few-rows kernel: a cluster takes an item up to these
constexpr double kOwnList = 12e6, kRowJoin = 6e3;         // many-rows kernel: ... as much as joining all rows, and one row

struct Lists {
    // items of the own keys
    bool tiles;                          // many-rows kernel
    int groups;                          // ... 128-row groups of an item
    int tok;                             // ... tokens of a group
    int nr;                              // few-rows kernel: 8-row groups of an item
    bool whole;                          // ... a CTA takes an item
    int split;                           // few-rows kernel: CTAs of the cluster that takes an item (0: a list)
    int M, rt, join;                     // M: rows of a partial result
    int64_t slots;
    // items of the prefix for the rows of all requests (many-rows kernel): in the same list when `tiles`
    bool pre;
    int pre_groups, pre_tok, pre_unit, pre_M, pre_items_rt;
    int64_t pre_slots;
};

// CTAs of the many-rows kernel at a time: one per SM, of one row group two.
int tile_workers(int sms, int groups) { return std::min(sms, kMaxTileWorkers) * (3 - groups); }

// Whether the many-rows kernel gives each CTA an item of up to `tiles` tiles.
bool whole_items(int64_t items, int64_t tiles, int groups, int workers) {
    return 5 * items <= 13 * (int64_t)workers && tiles <= 16 * groups &&
           tiles * groups * (2 * (int64_t)workers - items) <= 24 * (int64_t)workers;
}

// CTAs of a cluster that takes an item of up to `steps` steps whole; 0: the list.
int whole_split(int64_t items, int64_t steps, int sms) {
    int split = 0;
    if (items > (int64_t)kWholeItems * sms) return 0;
    int64_t least = kWholeSteps + 1;
    // Clusters do not fill a GPU to the last SM: 304 CTAs in fours take 9.3 us
    // where 152 in pairs take 5.8, 288 in fours 6.4.
    for (int j = 0; j < 4 && (j == 0 || (items << j) * 10 <= 19 * sms); ++j) {
        const int64_t cost = ceil_div(steps, kRowWarps << j) + (j > 0 ? j + 1 : 0);
        if (cost < least) {
            least = cost;
            split = 1 << j;
        }
    }
    return split;
}

// own_keys, pre_keys: by the table widths.  What a workspace has to hold does not
// depend on own_keys or sms.
Lists make_lists(int B, int Hkv, int G, int Nq, int D, int64_t own_keys, int64_t pre_keys, int sms) {
    Lists x{};
    const int64_t rows = (int64_t)Nq * G;
    x.tiles = rows > kFewRows && G <= 128;
    if (x.tiles && B > 1 && rows <= 64) {
        const int64_t tiles = ceil_div(pre_keys, 128), sets = ceil_div(B, 128 / rows);
        const double saved = (double)Hkv * ((double)B * tiles - (double)sets * (tiles + 3)) * 128 * D * 4;
        x.pre = saved > kOwnList + kRowJoin * (double)B * Hkv * rows;
    }
    if (!x.tiles) x.pre = rows <= kFewRows && B > 1 && (double)B * Hkv * pre_keys * D * 4 > (double)kReadAgain;
    if (x.pre) {
        x.pre_unit = (int)rows;
        x.pre_tok = 128 / x.pre_unit;
        x.pre_groups = x.tiles || B <= x.pre_tok ? 1 : 2;
        x.pre_M = 128 * x.pre_groups;
        x.pre_items_rt = (int)ceil_div(B, x.pre_tok * x.pre_groups);
        x.pre_slots = (int64_t)Hkv * x.pre_items_rt + kMaxTileWorkers * (3 - x.pre_groups);
    }
    if (x.tiles) {
        x.tok = 128 / G;
        if (x.pre) {
            x.groups = 1;
            x.M = (int)rows;
            x.rt = 1;
            x.slots = (int64_t)B * Hkv + 2 * kMaxTileWorkers;
            return x;
        }
        const int64_t tiles = ceil_div(own_keys, 128) + ceil_div(pre_keys, 128);
        const int workers = tile_workers(sms, 1);
        const int64_t items = (int64_t)B * Hkv * ceil_div(Nq, x.tok);      // of one group
        x.groups = Nq <= x.tok || ((items <= workers || tiles <= 4) && whole_items(items, tiles, 1, workers)) ? 1 : 2;
        x.M = 128 * x.groups;
        x.rt = (int)ceil_div(Nq, x.tok * x.groups);
        x.join = pre_keys > 0;
        x.whole = whole_items((int64_t)B * Hkv * x.rt, tiles, x.groups, tile_workers(sms, x.groups));
        x.slots = 2 * kMaxTileWorkers * (3 - x.groups);
        return x;
    }
    x.nr = rows <= 8 ? 1 : 2;                             // more than 16 rows: several sets
    x.M = 8 * x.nr;
    x.rt = (int)ceil_div(rows, x.M);
    x.slots = (int64_t)B * Hkv * x.rt + kMaxRowWorkers;
    x.join = pre_keys > 0 && !x.pre;
    if (!x.pre) x.split = whole_split((int64_t)B * Hkv * x.rt, ceil_div(own_keys, kStep) + ceil_div(pre_keys, kStep), sms);
    return x;
}

// Each array of the workspace begins on 16 bytes.
size_t padded(size_t n) { return (n + 15) / 16 * 16; }
size_t slot_bytes(int64_t slots, int M, int D) { return (size_t)slots * M * D * 4 + padded((size_t)slots * M * 8); }
size_t lists_bytes(const Lists& x, int B, int D) {
    const size_t index = x.tiles && !x.pre ? (size_t)2 * kMaxTileWorkers * sizeof(PagedCut) : padded(((size_t)B * x.rt + 1) * 4);
    return slot_bytes(x.slots, x.M, D) + slot_bytes(x.pre_slots, x.pre_M, D) + index;
}

int check_batch(int B, int H, int Hkv, int Nq, int D) {
    if (B <= 0 || H <= 0 || Hkv <= 0 || Nq <= 0 || H % Hkv != 0) return SAGE_ERR_ARG;
    if (B > 65535 || H > 65535 || Nq > (1 << 24)) return SAGE_ERR_ARG;
    if (D != 64 && D != 128) return SAGE_ERR_UNSUPPORTED;
    // row numbers stay in int
    if ((int64_t)B * Nq * (H / Hkv) > INT32_MAX / 2 || (int64_t)H * Nq > INT32_MAX / 2) return SAGE_ERR_UNSUPPORTED;
    return SAGE_OK;
}

int sm_count() {
    static int n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (n[dev] == 0 && cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n[dev];
}

// Join after a list of items of M rows and TK-key tiles.
template <int D, int M, int TK>
cudaError_t launch_join(const PagedParams& p, cudaStream_t s) {
    static bool ready8[64] = {}, ready1[64] = {};
    // Rows are few: eight warps share the parts of one, else a warp takes a row
    // (8 KV heads x 3 rows of 152 parts each: 4.2 against 13.6 us).
    const int64_t rows = (int64_t)p.H * p.Nq;
    if (rows * p.B <= 1024)
        return launch_pdl(paged_join_kernel<D, M, TK, 8>, dim3((unsigned)rows, (unsigned)p.B), dim3(256), 0, s, 1, true, ready8, p);
    return launch_pdl(paged_join_kernel<D, M, TK, 1>, dim3((unsigned)ceil_div(rows, 8), (unsigned)p.B), dim3(256), 0, s, 1, true,
                      ready1, p);
}

template <int D, int NR>
cudaError_t launch_rows(const PagedParams& p, cudaStream_t s) {
    if (p.split > 0) {
        static bool whole_ready[64] = {};
        return launch_pdl(paged_rows_kernel<D, NR, true>, dim3((unsigned)(p.B * p.rt * p.Hkv * p.split)), dim3(kRowWarps * 32),
                          RowsShape<D>::kSmem, s, p.split, true, whole_ready, p);
    }
    static bool ready[64] = {};
    const cudaError_t e = launch_pdl(paged_rows_kernel<D, NR, false>, dim3((unsigned)(p.workers / kRowWarps)), dim3(kRowWarps * 32),
                                     RowsShape<D>::kSmem, s, 1, true, ready, p);
    return e != cudaSuccess ? e : launch_join<D, 8 * NR, kStep>(p, s);
}
cudaError_t launch_rows(const PagedParams& p, int D, int nr, cudaStream_t s) {
    if (D == 64) return nr == 1 ? launch_rows<64, 1>(p, s) : launch_rows<64, 2>(p, s);
    return nr == 1 ? launch_rows<128, 1>(p, s) : launch_rows<128, 2>(p, s);
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_paged_workspace(int B, int H, int Hkv, int Nq, int D, size_t* bytes) {
    if (bytes == nullptr) return SAGE_ERR_ARG;
    const int rc = check_batch(B, H, Hkv, Nq, D);
    if (rc != SAGE_OK) return rc;
    // a prefix of any length may come: the form with a list of its own needs the most
    *bytes = lists_bytes(make_lists(B, Hkv, H / Hkv, Nq, D, 0, INT32_MAX, 0), B, D);
    const size_t alone = lists_bytes(make_lists(B, Hkv, H / Hkv, Nq, D, 0, 0, 0), B, D);
    if (alone > *bytes) *bytes = alone;
    return SAGE_OK;
}

int sage_attn_paged(const sage_tensor* q, const sage_tensor* o, const sage_page_cache* cache, int B, int H, int Nq,
                    const int32_t* q_len, const int32_t* table, int64_t table_stride, int table_width,
                    const int32_t* kv_len, const int32_t* prefix_table, int prefix_width, const int32_t* prefix_len,
                    float sm_scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_page_cache(cache);
    if (rc != SAGE_OK) return rc;
    const int D = cache->D;
    if ((rc = check_batch(B, H, cache->heads, Nq, D)) != SAGE_OK) return rc;
    for (const sage_tensor* t : {q, o}) {
        if ((rc = check_view(t)) != SAGE_OK) return rc;
        // rows apart (no broadcast axis), and byte strides that a tensor map holds
        if ((B > 1 && t->stride_b < D) || (H > 1 && t->stride_h < D) || (Nq > 1 && t->stride_n < D))
            return SAGE_ERR_UNSUPPORTED;
        for (int64_t st : {t->stride_b, t->stride_h, t->stride_n})
            if (st >= (int64_t(1) << 38)) return SAGE_ERR_UNSUPPORTED;
    }
    if (table_width < 0 || prefix_width < 0 || (table_width > 0 && table == nullptr) ||
        (prefix_width > 0 && prefix_table == nullptr) || table_stride < 0)
        return SAGE_ERR_ARG;
    const int64_t own_keys = (int64_t)table_width * cache->page_size;
    const int64_t pre_keys = (int64_t)prefix_width * cache->page_size;
    if (own_keys > INT32_MAX - 256 || pre_keys > INT32_MAX - 256) return SAGE_ERR_UNSUPPORTED;
    const int sms = sm_count();
    const Lists x = make_lists(B, cache->heads, H / cache->heads, Nq, D, own_keys, pre_keys, sms);
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < lists_bytes(x, B, D)) return SAGE_ERR_ARG;
    // list positions and slot numbers stay in int
    const int tk = x.tiles ? 128 : kStep;
    const int64_t tiles = (int64_t)B * cache->heads * x.rt * ((own_keys + (x.join ? pre_keys : 0)) / tk + 6) +
                          (int64_t)cache->heads * x.pre_items_rt * (pre_keys / tk + 6);
    if (tiles > INT32_MAX / 2 || x.slots + x.pre_slots > INT32_MAX / 2) return SAGE_ERR_UNSUPPORTED;

    PagedParams p{};
    p.status = device_status_ptr();
    if (p.status == nullptr || sms == 0) return SAGE_ERR_LAUNCH;
    CUtensorMap mq, mqp, mk, mv;
    if (x.tiles || x.pre) {
        // q in boxes of whole tokens; for the prefix's items, of whole requests
        const int heads = H / cache->heads;
        if ((x.tiles && (rc = encode_rows(&mq, *q, D, H, Nq, B, heads, x.tok, 1)) != SAGE_OK) ||
            (x.pre && (rc = encode_rows(&mqp, *q, D, H, Nq, B, heads, Nq, x.pre_tok)) != SAGE_OK) ||
            (rc = encode_pages(&mk, cache->k, D, cache->page_size, cache->heads, cache->num_pages)) != SAGE_OK ||
            (rc = encode_pages(&mv, cache->v, D, cache->page_size, cache->heads, cache->num_pages)) != SAGE_OK)
            return rc;
        if (!x.tiles) mq = mqp;
        if (!x.pre) mqp = mq;
        p.fault_mode = take_fault_mode();
    }
    p.q = static_cast<const uint16_t*>(q->ptr);
    p.o = static_cast<uint16_t*>(const_cast<void*>(o->ptr));
    p.k = static_cast<const uint16_t*>(cache->k.ptr);
    p.v = static_cast<const uint16_t*>(cache->v.ptr);
    p.qsb = q->stride_b; p.qsh = q->stride_h; p.qsn = q->stride_n;
    p.osb = o->stride_b; p.osh = o->stride_h; p.osn = o->stride_n;
    p.ksp = cache->k.stride_b; p.ksh = cache->k.stride_h; p.kst = cache->k.stride_n;
    p.vsp = cache->v.stride_b; p.vsh = cache->v.stride_h; p.vst = cache->v.stride_n;
    p.q_len = q_len; p.kv_len = kv_len; p.prefix_len = prefix_len;
    p.table = table; p.table_stride = table_stride; p.ptable = prefix_table;
    p.B = B; p.H = H; p.Hkv = cache->heads; p.G = H / cache->heads; p.Nq = Nq;
    p.W = table_width; p.Wp = prefix_width;
    p.num_pages = cache->num_pages; p.page = cache->page_size;
    p.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
    p.causal = causal != 0;
    const double scale = sm_scale > 0.f ? (double)sm_scale : 1.0 / std::sqrt((double)D);
    p.sc = (float)(scale * (1.0 / std::log(2.0)));
    p.rt = x.rt; p.join = x.join;
    p.tok = x.tok; p.part_m = x.M;
    p.by_G = make_fast_div(p.G);
    p.by_rt = make_fast_div(x.rt);
    char* w = static_cast<char*>(workspace);
    auto take = [&](size_t n) { char* at = w; w += padded(n); return at; };
    p.part_o = reinterpret_cast<float*>(take((size_t)x.slots * x.M * D * 4));
    p.part_ml = reinterpret_cast<float2*>(take((size_t)x.slots * x.M * 8));
    if (x.pre) {
        p.pre_o = reinterpret_cast<float*>(take((size_t)x.pre_slots * x.pre_M * D * 4));
        p.pre_ml = reinterpret_cast<float2*>(take((size_t)x.pre_slots * x.pre_M * 8));
        p.pre_unit = x.pre_unit;
        p.by_pre_unit = make_fast_div(x.pre_unit);
    }
    if (x.tiles && !x.pre) p.cuts = reinterpret_cast<PagedCut*>(w);
    else p.start = reinterpret_cast<int32_t*>(w);
    p.pre_items_rt = x.pre_items_rt; p.pre_m = x.pre_M; p.pre_tok = x.pre_tok;
    p.pre_workers = tile_workers(sms, x.pre_groups);
    p.whole = x.whole; p.split = x.split;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    int launches = 0;
    if (x.tiles) {
        p.workers = x.whole ? B * cache->heads * x.rt : tile_workers(sms, x.groups);
        if (x.pre) p.pre_rt = x.pre_items_rt;
        e = launch_paged_tiles(p, D, x.groups, mq, mqp, mk, mv, s);
        if (e == cudaSuccess && x.pre) e = D == 64 ? launch_join<64, 128, 128>(p, s) : launch_join<128, 128, 128>(p, s);
        launches = p.whole ? 1 : 2;
    } else {
        if (x.pre) {
            PagedParams pp = p;
            pp.start = nullptr;
            pp.rt = 0; pp.pre_rt = x.pre_items_rt; pp.workers = p.pre_workers;
            if (launch_paged_tiles(pp, D, x.pre_groups, mq, mqp, mk, mv, s) != cudaSuccess) return SAGE_ERR_LAUNCH;
            ++launches;
            p.beside = 1;
        }
        p.workers = std::min(2 * sms, kMaxRowWorkers / kRowWarps) * kRowWarps;
        e = launch_rows(p, D, x.nr, s);
        launches += p.split > 0 ? 1 : 2;
    }
    if (e != cudaSuccess) return SAGE_ERR_LAUNCH;
    set_last_launch_count(launches);
    return SAGE_OK;
}

}  // extern "C"
