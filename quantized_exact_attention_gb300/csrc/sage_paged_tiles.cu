// sage_paged_tiles.cu - attention over a page cache for many query rows, on
// the tcgen05 tensor cores.
//
// One persistent CTA per SM is one worker of the list of sage_paged_sched.cuh
// with 128-key tiles.  Two groups of 128 query rows take turns at the tensor
// core: while one group's scores go through the softmax, the other group's
// products run.  A "unit" is one group's S = Q K^T and O += P V of one tile.
//   plain form (M = 256 rows of an item): both groups see every tile, group X
//     holds rows [128 X, 128 X + 128);
//   split form (M = 128): both groups hold the same rows and take every other
//     tile; their results join in shared memory when the item ends.  It keeps
//     two units in flight where there are only rows for one.
//
// Warp roles (320 threads):
//   warps 0-3, 4-7  softmax of group 0 and 1, one thread per row: S from tensor
//                   memory, mask, online maximum and sum, P in BF16 over the
//                   columns of its S; at an item's ends Q into shared memory
//                   and the output from tensor memory
//   warp 8          TMA producer: the pages of a K and of a V tile through
//                   rings of stages; it alone walks the list and leaves a note
//                   for each tile
//   warp 9          tensor-memory allocator and single-thread tcgen05 issuer
// Tensor memory: S/P of group X at column 128 X, O of group X at 256 + 128 X.
//
// The reference of the exponentials follows the row maximum lazily: O is
// rescaled only when the maximum has grown by more than 2^8 since the last
// rescale.  The weights then reach 2^8 at most, which BF16 holds at the same
// relative error, and the rescale (a round trip of O through registers)
// almost never runs.
//
// Waits are bounded as in sage_attn.cu: one that runs out records
// SAGE_ERR_TIMEOUT, raises the CTA's abort flag, and every role leaves its
// loop, lets its copies and products land, and returns.
#include "sage_gb300.h"
#include "sage_internal.h"
#include "sage_paged.h"
#include "sage_paged_sched.cuh"
#include "sage_ptx.cuh"

namespace sage {
namespace {

constexpr int kTileThreads = 320;
constexpr int kWarpLoad = 8;
constexpr int kWarpIssue = 9;
constexpr int kNotes = 8;
constexpr float kLazy = 8.f;                              // log2 of the weights' bound
constexpr uint32_t kBlk = 128 * 128;                      // 128 rows x 64 channels
constexpr uint32_t TM_O = 256;

enum TileRole { R_ROWS = 6, R_LOAD = 7, R_ISSUE = 8 };

// What the loader says about a tile.
struct TileNote {
    int b, h, rt;
    int key0, nkeys;
    int n, len;                                           // the request's query tokens and own keys
    int slot;                                             // of a partial result
    int flags;
    int pad[3];
};
enum { N_FIRST = 1, N_LAST = 2, N_OWN = 4, N_WHOLE = 8 };  // of its item in this worker; own keys; item not shared

template <int D, bool kSplit>
struct TilesShape {
    static constexpr int M = kSplit ? 128 : 256;
    static constexpr int kNB = D / 64;                    // 64-channel blocks of a row
    static constexpr uint32_t kTile = kNB * kBlk;         // bytes of a K (or V) tile
    static constexpr int kNS = D == 128 ? 2 : 4;          // K and V stages
    static constexpr uint32_t OFF_Q = 0;                  // two groups' Q; split: one Q, later the join buffer
    static constexpr uint32_t OFF_K = 2 * kTile;
    static constexpr uint32_t OFF_V = OFF_K + kNS * kTile;
    static constexpr uint32_t OFF_BAR = OFF_V + kNS * kTile;
    // barriers
    static constexpr int B_Q = 0, B_ITEM = 1, B_JOIN = 2, B_ODONE = 3, B_DRAIN = 4, B_S = 5, B_P = 7;
    static constexpr int B_KF = 9, B_KE = B_KF + kNS, B_VF = B_KE + kNS, B_VE = B_VF + kNS, B_NOTE = B_VE + kNS;
    static constexpr int kBars = B_NOTE + kNotes;
    static constexpr uint32_t OFF_NOTE = OFF_BAR + (kBars * 8 + 15) / 16 * 16;
    static constexpr uint32_t OFF_ML = OFF_NOTE + kNotes * sizeof(TileNote);      // float2 [128]
    static constexpr uint32_t OFF_SCAN = OFF_ML + 128 * 8;                        // int [320 + 16]
    static constexpr uint32_t OFF_TMEM = OFF_SCAN + (kTileThreads + 16) * 4;
    static constexpr uint32_t OFF_ABORT = OFF_TMEM + 16;
    static constexpr uint32_t kSmem = OFF_ABORT + 16 + 1024;                      // + alignment slack
};

// Instruction descriptor: BF16 operands, FP32 accumulator; B either K-major
// (K: a row is a key) or N-major (V: a row is a key, channels contiguous).
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t N, bool b_n_major) {
    return idesc_f32acc(1u, 128u, N) | (b_n_major ? 1u << 16 : 0u);
}
// N-major operand in the 128-byte swizzle layout: 64-channel blocks kBlk
// apart (leading offset), groups of 8 keys 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t sdesc_n_major(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(kBlk >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
// D[tmem] (+)= A[tmem] * B[smem], 16-bit inputs, FP32 accumulate.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// Whether the phase with the given parity is complete; never suspends.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(kTileThreads, 1)
paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ PagedParams p) {
    using L = TilesShape<D, kSplit>;
    constexpr int M = L::M, NS = L::kNS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t sbase = (raw_base + 1023u) & ~1023u;
    uint8_t* sgen = smem_raw + (sbase - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const PagedSched<M, 128> sched(p);
    int* chunk = reinterpret_cast<int*>(sgen + L::OFF_SCAN);
    const int total = paged_scan<M, 128, kTileThreads>(sched, chunk, chunk + kTileThreads, p.start != nullptr && blockIdx.x == 0);
    const int per = sched.per_worker(total);
    const int worker = blockIdx.x;
    if ((int64_t)worker * per >= total) return;
    const int t0 = worker * per;
    const int count = min(per, total - t0);

    auto bar = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)i; };
    TileNote* notes = reinterpret_cast<TileNote*>(sgen + L::OFF_NOTE);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sgen + L::OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::OFF_ABORT);
    auto fail = [&](int role, int tile) {
        *abort_flag = 1;
        if (atomicCAS(p.status, 0, -4 /* SAGE_ERR_TIMEOUT */) == 0) {
            p.status[1] = (int)blockIdx.x;
            p.status[2] = role;
            p.status[3] = tile;
        }
    };

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(bar(L::B_Q), 256);
        mbar_init(bar(L::B_ITEM), 256);
        mbar_init(bar(L::B_JOIN), 128);
        mbar_init(bar(L::B_ODONE), 1);
        mbar_init(bar(L::B_DRAIN), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::B_S + i), 1);
            mbar_init(bar(L::B_P + i), 128);
        }
        for (int i = 0; i < 4 * NS; ++i) mbar_init(bar(L::B_KF + i), 1);
        for (int i = 0; i < kNotes; ++i) mbar_init(bar(L::B_NOTE + i), 1);
        fence_mbar_init();
    }
    if (warp == kWarpIssue) {
        tmem_alloc(sbase + L::OFF_TMEM, 512);
        tmem_relinquish();
    }
    if (warp == kWarpLoad && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 8) {
        // ===================================================== softmax
        const int X = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + 128u * X, tO = tmem + lane_base + TM_O + 128u * X;
        float2* ml_s = reinterpret_cast<float2*>(sgen + L::OFF_ML);
        float m = -INFINITY, l = 0.f;                      // reference of the exponentials (log2 domain), sum
        bool fresh = true;                                // no tile of this item yet: O holds nothing
        bool valid = false, active = false;               // this row exists; some row of this warp does
        int rb = 0, ri = 0, rh = 0, lim_own = 0;
        int units = 0, items = 0;
        bool ok = true;
        for (int t = 0; t < count && ok; ++t) {
            if (!mbar_wait_warp(bar(L::B_NOTE + t % kNotes), (t / kNotes) & 1, abort_flag)) {
                if (lane == 0) fail(R_ROWS, t);
                break;
            }
            const TileNote& nt = notes[t % kNotes];
            const int flags = nt.flags;
            if (flags & N_FIRST) {
                // Both groups have left the item before: its products are done
                // (each waited for them) and the join buffer has been read.
                mbar_arrive(bar(L::B_ITEM));
                PagedPlace x{};
                x.b = nt.b; x.h = nt.h; x.rt = nt.rt; x.n = nt.n; x.len = nt.len;
                valid = paged_row(sched, x, kSplit ? row : X * 128 + row, rb, ri, rh);
                active = __any_sync(0xffffffffu, valid);
                lim_own = nt.len;
                if (p.causal && nt.b >= 0) lim_own = min(nt.len, nt.len - nt.n + ri + 1);
                m = -INFINITY; l = 0.f; fresh = true;
                // Q rows in the K-major 128-byte swizzle; split: each group half of the channels
                constexpr int kC = kSplit ? D / 16 : D / 8;
                const int c0 = kSplit ? X * kC : 0;
                const uint16_t* qp = p.q + (valid ? rb * p.qsb + rh * p.qsh + ri * p.qsn : 0);
                uint4 qv[kC];
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    qv[c] = valid ? __ldg(reinterpret_cast<const uint4*>(qp) + c0 + c) : make_uint4(0, 0, 0, 0);
                if (!mbar_wait_warp(bar(L::B_ITEM), items & 1, abort_flag)) {
                    if (lane == 0) fail(R_ROWS, t);
                    break;
                }
                uint8_t* qs = sgen + L::OFF_Q + (kSplit ? 0 : X * L::kTile) + row * 128;
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const int cc = c0 + c;
                    *reinterpret_cast<uint4*>(qs + (cc >> 3) * kBlk + (((cc & 7) ^ (row & 7)) << 4)) = qv[c];
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(L::B_Q));
            }
            if (!kSplit || (t & 1) == X) {
                const int nkeys = nt.nkeys;
                int lim = nkeys;
                if (flags & N_OWN) lim = min(lim, lim_own - nt.key0);
                if (!mbar_wait_warp(bar(L::B_S + X), units & 1, abort_flag)) {
                    if (lane == 0) fail(R_ROWS, t);
                    break;
                }
                ++units;
                tc_fence_after();
                if (active) {
                    uint32_t s[4][32];
                    float mx0, mx1;
                    tmem_ld64_max(tS, s[0], s[1], mx0);
                    tmem_ld64_max(tS + 64, s[2], s[3], mx1);
                    tmem_wait_ld();
                    float mx = fmaxf(mx0, mx1);
                    if (!__all_sync(0xffffffffu, lim >= 128)) {
                        mx = -INFINITY;
#pragma unroll
                        for (int a = 0; a < 4; ++a)
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (a * 32 + i >= lim) s[a][i] = 0xFF800000u;    // -inf
                                mx = fmaxf(mx, __uint_as_float(s[a][i]));
                            }
                    }
                    const float mt = mx * p.sc;
                    const bool grow = mt > m + kLazy;      // also the first visible key: m = -inf
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mn = grow ? mt : m;
                        const float f = grow ? ex2_approx(m - mn) : 1.f;
                        l *= f;
                        m = mn;
                        if (!fresh) {
                            // the products of this group's earlier tiles are done:
                            // its scores were issued behind them
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(tO + c * 32, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st32(tO + c * 32, o);
                            }
                        }
                    }
                    const float neg = m == -INFINITY ? 0.f : -m;
                    float l0 = 0.f, l1 = 0.f;
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int b = a * 64 + 2 * i;
                            float x0, x1;
                            fma2_bc(x0, x1, __uint_as_float(s[b / 32][b % 32]), __uint_as_float(s[b / 32][b % 32 + 1]),
                                    p.sc, neg);
                            x0 = ex2_approx(x0);
                            x1 = ex2_approx(x1);
                            add2(l0, l1, x0, x1);
                            w[i] = pack2(x0, x1);
                        }
                        tmem_st32(tS + a * 32, w);
                    }
                    l += l0 + l1;
                    tmem_wait_st();
                }
                fresh = false;
                tc_fence_before();
                // V rows behind the last key: whatever they hold times a weight
                // of 0 must be 0 (kSplit or not, before the first product reads them)
                if (nkeys < 128 && (kSplit || X == 0)) {
                    if (!mbar_wait_warp(bar(L::B_VF + t % NS), (t / NS) & 1, abort_flag)) {
                        if (lane == 0) fail(R_ROWS, t);
                        break;
                    }
                    if (row >= nkeys) {
                        uint8_t* vr = sgen + L::OFF_V + (t % NS) * L::kTile + row * 128;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4*>(vr + (c >> 3) * kBlk + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                mbar_arrive(bar(L::B_P + X));
            }
            if (flags & N_LAST) {
                if (!mbar_wait_warp(bar(L::B_ODONE), items & 1, abort_flag)) {
                    if (lane == 0) fail(R_ROWS, t);
                    break;
                }
                tc_fence_after();
                float fa = 1.f, fb = 0.f;                 // weights of this group's and the other group's O
                uint8_t* jr = sgen + L::OFF_Q + row * (D * 4);
                constexpr int kSw = D / 4 - 1;            // 16-byte chunks of a join row, less one
                if constexpr (kSplit) {
                    if (X == 1) {
                        ml_s[row] = make_float2(m, l);
                        if (active && !fresh) {
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(tO + c * 32, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    *reinterpret_cast<uint4*>(jr + (((c * 8 + i) ^ (row & kSw)) << 4)) =
                                        make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            }
                        }
                        mbar_arrive(bar(L::B_JOIN));
                    } else {
                        if (!mbar_wait_warp(bar(L::B_JOIN), items & 1, abort_flag)) {
                            if (lane == 0) fail(R_ROWS, t);
                            break;
                        }
                        const float2 other = ml_s[row];
                        const float mn = fmaxf(m, other.x);
                        const float ms = mn == -INFINITY ? 0.f : mn;
                        fa = ex2_approx(m - ms);
                        fb = ex2_approx(other.x - ms);
                        l = l * fa + other.y * fb;
                        m = mn;
                    }
                }
                if (active && (!kSplit || X == 0)) {
                    const bool whole = (flags & N_WHOLE) != 0;
                    const float inv = whole ? (l == 0.f ? 0.f : __fdiv_rn(1.f, l)) : 1.f;
                    const int r = kSplit ? row : X * 128 + row;
                    const int64_t slot_row = (int64_t)nt.slot * M + r;
                    if (valid && !whole) p.part_ml[slot_row] = make_float2(m, l);
                    uint16_t* dst = p.o + rb * p.osb + rh * p.osh + (int64_t)ri * p.osn;
                    float* part = p.part_o + slot_row * D;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + c * 32, o);
                        tmem_wait_ld();
                        float x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]);
                        if constexpr (kSplit) {
                            // a group without a tile, or without a visible key, adds nothing
                            // (its O may hold anything)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 y = *reinterpret_cast<const float4*>(jr + (((c * 8 + i) ^ (row & kSw)) << 4));
                                const float yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[4 * i + e] = (fa == 0.f ? 0.f : x[4 * i + e] * fa) + (fb == 0.f ? 0.f : yy[e] * fb);
                            }
                        }
                        if (valid && whole) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[e] = pack2(x[8 * i + 2 * e] * inv, x[8 * i + 2 * e + 1] * inv);
                                reinterpret_cast<uint4*>(dst)[c * 4 + i] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else if (valid) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                reinterpret_cast<float4*>(part)[c * 8 + i] =
                                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();
                ++items;
            }
        }
    } else if (warp == kWarpLoad) {
        // ===================================================== TMA producer
        PagedPlace at = paged_find<M, 128, kTileThreads>(sched, chunk, t0);
        const int per_tile = 128 >> p.page_shift;         // pages of a whole tile
        PagedSpan span = paged_span(sched, at);
        bool first = true;
        int run0 = at.tile;                               // the item's first tile in this worker
        auto page_of = [&](const PagedSpan& sp, const PagedPlace& x) -> int {
            if (lane >= per_tile || (lane << p.page_shift) >= sp.nkeys) return 0;
            const int j = (sp.key0 >> p.page_shift) + lane;
            return sp.own ? __ldg(p.table + (int64_t)x.b * p.table_stride + j) : __ldg(p.ptable + j);
        };
        int page = page_of(span, at);
        int loaded_k = 0, loaded_v = 0;                   // tiles whose copies were issued
        bool ok = true;
        for (int t = 0; t < count; ++t) {
            const int st = t % NS, ph = (t / NS) & 1;
            const bool mine = lane < per_tile && (lane << p.page_shift) < span.nkeys;
            const uint32_t bytes = (uint32_t)((span.nkeys + p.page - 1) >> p.page_shift) * (uint32_t)(p.page * 128 * L::kNB);
            const uint32_t off = (uint32_t)(lane * p.page) * 128u;
            // a page outside the cache: the copy reads zeros there
            if (mine && (unsigned)page >= (unsigned)p.num_pages && atomicCAS(p.status, 0, kErrPage) == 0) p.status[3] = page;
            if (t >= NS && !mbar_wait_warp(bar(L::B_KE + st), ph ^ 1, abort_flag)) { ok = false; break; }
            if (lane == 0) {
                TileNote& nt = notes[t % kNotes];
                const bool last = t + 1 == count || at.tile + 1 == at.ntiles;
                nt.b = at.b; nt.h = at.h; nt.rt = at.rt;
                nt.key0 = span.key0; nt.nkeys = span.nkeys;
                nt.n = at.n; nt.len = at.len;
                nt.slot = p.pre_rt > 0 ? worker + at.item : 2 * worker + (run0 == 0 ? 1 : 0);
                nt.flags = (first ? N_FIRST : 0) | (last ? N_LAST : 0) | (span.own ? N_OWN : 0) |
                           (p.pre_rt == 0 && run0 == 0 && at.tile + 1 == at.ntiles ? N_WHOLE : 0);
                mbar_arrive(bar(L::B_NOTE + t % kNotes));
                mbar_arrive_expect_tx(bar(L::B_KF + st), bytes);
            }
            __syncwarp();
            if (mine) {
#pragma unroll
                for (int hb = 0; hb < L::kNB; ++hb)
                    tma_load_4d(sbase + L::OFF_K + st * L::kTile + hb * kBlk + off, &tm_k, hb * 64, 0, at.h, page,
                                bar(L::B_KF + st));
            }
            loaded_k = t + 1;
            if (t >= NS && !mbar_wait_warp(bar(L::B_VE + st), ph ^ 1, abort_flag)) { ok = false; break; }
            if (lane == 0) mbar_arrive_expect_tx(bar(L::B_VF + st), bytes);
            __syncwarp();
            if (mine && p.fault_mode != 1) {
#pragma unroll
                for (int hb = 0; hb < L::kNB; ++hb)
                    tma_load_4d(sbase + L::OFF_V + st * L::kTile + hb * kBlk + off, &tm_v, hb * 64, 0, at.h, page,
                                bar(L::B_VF + st));
            }
            loaded_v = t + 1;
            if (t + 1 < count) {
                const int item = at.item;
                paged_next(sched, at);
                first = at.item != item;
                if (first) run0 = at.tile;
                span = paged_span(sched, at);
                page = page_of(span, at);
            }
        }
        if (!ok && lane == 0) fail(R_LOAD, loaded_v);
        __syncwarp();
        // every copy issued lands before the CTA may exit
        const int zero = 0;
        for (int i = 0; i < NS; ++i) {
            int tk = loaded_k - 1 - i, tv = loaded_v - 1 - i;
            if (tk >= 0) mbar_wait_warp(bar(L::B_KF + tk % NS), (tk / NS) & 1, &zero);
            if (tv >= 0 && p.fault_mode != 1) mbar_wait_warp(bar(L::B_VF + tv % NS), (tv / NS) & 1, &zero);
        }
    } else if (lane == 0) {
        // ===================================================== MMA issuer
        constexpr uint32_t kIdescQK = idesc_bf16(128, false);
        constexpr uint32_t kIdescPV = idesc_bf16(D, true);
        constexpr int kUnitsPerTile = kSplit ? 1 : 2;
        const uint64_t dQ = sdesc_sw128(sbase + L::OFF_Q);
        const uint64_t dK = sdesc_sw128(sbase + L::OFF_K);
        const uint64_t dV = sdesc_n_major(sbase + L::OFF_V);
        const int U = count * kUnitsPerTile;
        int s = 0, v = 0;                                 // next unit whose S, whose PV is issued
        int noted = 0;                                    // tiles whose note has been read
        uint32_t firsts = 0, lasts = 0;                   // their flags, bit tile % 32
        int items = 0;                                    // items whose first S has been issued
        uint32_t summed = 0;                              // bit X: group X has a product in this item
        bool ok = true;
        unsigned long long since = 0;
        uint32_t polls = 0;
        while (v < U) {
            bool moved = false;
            // S of unit s: at most two units ahead (its columns hold the P of
            // unit s - 2), and into a new item only when the item before it is
            // through (its Q is overwritten, and its output read, after that).
            if (s < U && s < v + 2) {
                const int t = s / kUnitsPerTile, st = t % NS;
                bool ready = true;
                if (t == noted) {
                    ready = mbar_test_wait(bar(L::B_KF + st), (t / NS) & 1);
                    if (ready) {
                        const int f = notes[t % kNotes].flags;
                        firsts = (firsts & ~(1u << (t & 31))) | ((f & N_FIRST ? 1u : 0u) << (t & 31));
                        lasts = (lasts & ~(1u << (t & 31))) | ((f & N_LAST ? 1u : 0u) << (t & 31));
                        ++noted;
                    }
                }
                const bool opens = ready && ((firsts >> (t & 31)) & 1u) && s % kUnitsPerTile == 0;
                if (opens) ready = v == s && mbar_test_wait(bar(L::B_Q), items & 1);
                if (ready) {
                    if (opens) ++items;
                    const int X = s & 1;
                    tc_fence_after();
                    const uint64_t a = dQ + (uint64_t)((kSplit ? 0 : X * L::kTile) >> 4);
                    const uint64_t b = dK + (uint64_t)((st * L::kTile) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t o = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
                        mma_f16_ss(tmem + 128u * X, a + o, b + o, kIdescQK, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(bar(L::B_S + X));
                    if (s % kUnitsPerTile == kUnitsPerTile - 1) mma_commit(bar(L::B_KE + st));
                    ++s;
                    moved = true;
                }
            }
            if (v < s) {
                const int t = v / kUnitsPerTile, st = t % NS, X = v & 1;
                if (mbar_test_wait(bar(L::B_P + X), (v >> 1) & 1) && mbar_test_wait(bar(L::B_VF + st), (t / NS) & 1)) {
                    tc_fence_after();
                    if (((firsts >> (t & 31)) & 1u) && v % kUnitsPerTile == 0) summed = 0;
                    const uint64_t b = dV + (uint64_t)((st * L::kTile) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_f16_ts(tmem + TM_O + 128u * X, tmem + 128u * X + kk * 8, b + (uint64_t)(kk * (2048 >> 4)),
                                   kIdescPV, kk > 0 || ((summed >> X) & 1u) ? 1u : 0u);
                    summed |= 1u << X;
                    if (v % kUnitsPerTile == kUnitsPerTile - 1) {
                        mma_commit(bar(L::B_VE + st));
                        if ((lasts >> (t & 31)) & 1u) mma_commit(bar(L::B_ODONE));
                    }
                    ++v;
                    moved = true;
                }
            }
            if (moved) {
                polls = 0;
            } else if ((++polls & 63u) == 0) {
                if (*abort_flag) { ok = false; break; }
                const unsigned long long now = globaltimer();
                if (polls == 64) since = now;
                else if (now - since > kWaitLimitNs) { ok = false; break; }
            }
        }
        if (!ok) fail(R_ISSUE, v);
        mma_commit(bar(L::B_DRAIN));                       // all products done before teardown
        const int zero = 0;
        mbar_wait(bar(L::B_DRAIN), 0, &zero);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpIssue) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Join the items that a worker boundary cuts (list without shared prefix
// items; whole items were written by the kernel above).  blockIdx.x + 1 is
// the boundary, blockIdx.y a group of 32 rows.
// ---------------------------------------------------------------------------
template <int D, int M>
__global__ void __launch_bounds__(256) paged_cuts_kernel(const PagedParams p) {
    constexpr int V = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedSched<M, 128> s(p);
    const int total = p.start[p.B];
    const int per = s.per_worker(total);
    const int w = blockIdx.x + 1;
    if ((int64_t)w * per >= total) return;
    const int pos = w * per;
    int lo = 0, hi = p.B - 1;                              // last request that starts at or before pos
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.start[mid] <= pos) lo = mid; else hi = mid - 1;
    }
    PagedPlace x{};
    x.b = lo;
    x.n = s.q_rows(lo);
    x.len = s.own_keys(lo);
    const int per_head = (p.start[lo + 1] - p.start[lo]) / p.Hkv;
    x.h = (pos - p.start[lo]) / per_head;
    int at = p.start[lo] + x.h * per_head, nt = 0;
    for (x.rt = 0; x.rt < p.rt; ++x.rt) {
        nt = s.item_tiles(x.n, x.len, x.rt);
        if (pos < at + nt) break;
        at += nt;
    }
    if (at >= pos || at / per != w - 1) return;            // the item starts here, or was cut before
    const int w1 = (at + nt - 1) / per;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = (int)blockIdx.y * 32 + k * 8 + warp;
        int b, i, hq;
        if (!paged_row(s, x, r, b, i, hq)) continue;
        float acc[V], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
        for (int ww = w - 1; ww <= w1; ++ww) {
            const int64_t q = (int64_t)(2 * ww + (ww == w - 1 ? 1 : 0)) * M + r;
            const float2 ml = __ldcg(p.part_ml + q);
            const float* src = p.part_o + q * D + lane;
            const float mn = fmaxf(m, ml.x);
            const float ms = mn == -INFINITY ? 0.f : mn;
            const float fa = ex2_approx(m - ms), fb = ex2_approx(ml.x - ms);
            l = l * fa + ml.y * fb;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = acc[v] * fa + __ldcg(src + 32 * v) * fb;
            m = mn;
        }
        const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
        uint16_t* dst = p.o + b * p.osb + hq * p.osh + (int64_t)i * p.osn + lane;
#pragma unroll
        for (int v = 0; v < V; ++v) dst[32 * v] = (uint16_t)pack2(acc[v] * inv, 0.f);
    }
}

template <int D, bool kSplit>
cudaError_t launch_one(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t s) {
    using L = TilesShape<D, kSplit>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(paged_tiles_kernel<D, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    paged_tiles_kernel<D, kSplit><<<ctas, kTileThreads, L::kSmem, s>>>(tk, tv, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.pre_rt == 0 && ctas > 1) {
        paged_cuts_kernel<D, L::M><<<dim3((unsigned)ctas - 1, L::M / 32), 256, 0, s>>>(p);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedParams& p, int D, bool split, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
    if (D == 64) return split ? launch_one<64, true>(p, tk, tv, p.workers, s) : launch_one<64, false>(p, tk, tv, p.workers, s);
    return split ? launch_one<128, true>(p, tk, tv, p.workers, s) : launch_one<128, false>(p, tk, tv, p.workers, s);
}

}  // namespace sage
