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
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax of group 0 and 1, one thread per row: S from tensor
//                   memory, mask, online maximum and sum, P in BF16 over the
//                   columns of its S; at an item's ends Q into shared memory
//                   and the output from tensor memory
//   warp 8          TMA producer: the pages of a K and of a V tile through
//                   rings of stages; it alone walks the list and leaves a note
//                   for each tile
//   warp 9          tensor-memory allocator; one thread issues S = Q K^T
//   warp 10         one thread issues O += P V
//   warp 11         idle; it completes the warpgroup whose registers go to the
//                   softmax (setmaxnreg: 2 x 128 x 224 + 128 x 56 = 384 x 168)
// Tensor memory: O of group X in the top 2 D columns, P of group X beside its
// S.  D = 128: [S 128 | P0 64 | P1 64 | O0 128 | O1 128], one S for both
// groups: a group loads its scores into registers at once and frees it, so the
// next scores are computed while both groups' exponentials run, and a group
// never waits for its own P V.  D = 64: [S0 128 | S1 128 | P0 | P1 | O0 | O1].
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

constexpr int kTileThreads = 384;
constexpr int kWarpLoad = 8;
constexpr int kWarpS = 9;
constexpr int kWarpPV = 10;
constexpr int kNotes = 8;
constexpr float kLazy = 8.f;                              // log2 of the weights' bound
constexpr uint32_t kBlk = 128 * 128;                      // 128 rows x 64 channels

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
    static constexpr int kSBufs = D == 128 ? 1 : 2;       // S buffers in tensor memory
    static constexpr uint32_t TM_P = 128 * kSBufs;        // + 64 X
    static constexpr uint32_t TM_O = TM_P + 128;          // + D X
    static constexpr uint32_t OFF_Q = 0;                  // two groups' Q; split: one Q, later the join buffer
    static constexpr uint32_t OFF_K = 2 * kTile;
    static constexpr uint32_t OFF_V = OFF_K + kNS * kTile;
    static constexpr uint32_t OFF_STAGE = OFF_V + kNS * kTile;                    // split: rows on their way out
    static constexpr uint32_t OFF_BAR = OFF_STAGE + (kSplit ? 4 * 4096 : 0);
    // barriers
    static constexpr int B_Q = 0, B_ITEM = 1, B_JOIN = 2, B_ODONE = 3, B_DRAIN = 4;
    static constexpr int B_S = 6, B_SFREE = 8, B_P = 10, B_PV = 12;               // one of each per group
    static constexpr int B_KF = 14, B_KE = B_KF + kNS, B_VF = B_KE + kNS, B_VE = B_VF + kNS, B_NOTE = B_VE + kNS;
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
// One elected lane of a converged warp issues; the operands are warp-uniform.
// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit inputs, FP32 accumulate.
__device__ __forceinline__ void mma_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// The same lane is elected each time, so it is the thread that issued the products.
__device__ __forceinline__ void commit_elect(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(bar) : "memory");
}
// The bounded wait of the hand-offs between softmax and issuers.  It polls with
// test_wait, which never suspends the warp (a suspended try_wait adds its
// wake-up to the hand-off), and looks at the clock only every 1,024 polls.
// All 32 lanes call it together.
__device__ __forceinline__ bool mbar_spin_warp(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
    unsigned long long t0 = 0;
    for (uint32_t i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (__all_sync(0xffffffffu, ok != 0)) return true;
        if ((i & 1023u) == 0) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
            const unsigned long long now = globaltimer();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xffffffffu, now - t0 > kWaitLimitNs)) return false;
        }
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Store kC 16-byte chunks of each lane's row (at base + at; at < 0: no row)
// through 32 staged rows of 128 bytes.  All 32 lanes call it together.
template <int kC, class T>
__device__ __forceinline__ void stage_out(uint8_t* stage, const uint32_t (&o)[32], int64_t at, T* base, int lane) {
#pragma unroll
    for (int i = 0; i < kC; ++i)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
            make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        const int r = i * (32 / kC) + lane / kC, c = lane % kC;
        const int64_t a = __shfl_sync(0xffffffffu, at, r);
        const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
        if (a >= 0) reinterpret_cast<uint4*>(base + a)[c] = w;
    }
    __syncwarp();
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::B_DRAIN + i), 1);
            mbar_init(bar(L::B_S + i), 1);
            mbar_init(bar(L::B_SFREE + i), 4);            // one arrival a warp
            mbar_init(bar(L::B_P + i), 4);
            mbar_init(bar(L::B_PV + i), 1);
        }
        for (int i = 0; i < 4 * NS; ++i) mbar_init(bar(L::B_KF + i), 1);
        for (int i = 0; i < kNotes; ++i) mbar_init(bar(L::B_NOTE + i), 1);
        fence_mbar_init();
    }
    if (warp == kWarpS) {
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int X = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + (L::kSBufs == 2 ? 128u * X : 0u);
        const uint32_t tP = tmem + lane_base + L::TM_P + 64u * X, tO = tmem + lane_base + L::TM_O + (uint32_t)D * X;
        float2* ml_s = reinterpret_cast<float2*>(sgen + L::OFF_ML);
        float m = -INFINITY, l = 0.f;                      // reference of the exponentials (log2 domain), sum
        bool fresh = true;                                // no tile of this item yet: O holds nothing
        bool valid = false, active = false;               // this row exists; some row of this warp does
        int rb = 0, ri = 0, rh = 0, lim_own = 0;
        int64_t o_at = -1;                                // offset of this row's output, -1: none
        int units = 0, items = 0;
        bool ok = true;
        for (int t = 0; t < count && ok; ++t) {
            if (!mbar_spin_warp(bar(L::B_NOTE + t % kNotes), (t / kNotes) & 1, abort_flag)) {
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
                // Q in the K-major 128-byte swizzle.  A warp fetches its 32 rows with
                // neighbouring lanes on neighbouring chunks of a row (one row a lane
                // would touch 32 lines with each load); split: each group half of
                // the channels.
                constexpr int kC = kSplit ? D / 16 : D / 8;           // 16-byte chunks of a row
                constexpr int kR = 32 / kC;                           // rows a load covers
                constexpr int kQ = kC < 8 ? kC : 8;                   // loads in flight
                const int c0 = kSplit ? X * kC : 0;
                const int64_t q_at = valid ? rb * p.qsb + rh * p.qsh + ri * p.qsn : -1;
                o_at = valid ? rb * p.osb + rh * p.osh + ri * p.osn : -1;
                if (!mbar_wait_warp(bar(L::B_ITEM), items & 1, abort_flag)) {
                    if (lane == 0) fail(R_ROWS, t);
                    break;
                }
                uint8_t* qs = sgen + L::OFF_Q + (kSplit ? 0 : X * L::kTile);
#pragma unroll 1
                for (int i0 = 0; i0 < kC; i0 += kQ) {
                    uint4 qv[kQ];
#pragma unroll
                    for (int i = 0; i < kQ; ++i) {
                        const int64_t at = __shfl_sync(0xffffffffu, q_at, (i0 + i) * kR + lane / kC);
                        qv[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.q + at) + c0 + lane % kC)
                                        : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < kQ; ++i) {
                        const int r = (warp & 3) * 32 + (i0 + i) * kR + lane / kC, c = c0 + lane % kC;
                        *reinterpret_cast<uint4*>(qs + (c >> 3) * kBlk + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = qv[i];
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(L::B_Q));
            }
            if (!kSplit || (t & 1) == X) {
                const int nkeys = nt.nkeys;
                int lim = nkeys;
                if (flags & N_OWN) lim = min(lim, lim_own - nt.key0);
                if (!mbar_spin_warp(bar(L::B_S + X), units & 1, abort_flag)) {
                    if (lane == 0) fail(R_ROWS, t);
                    break;
                }
                tc_fence_after();
                // Keys that some row of this warp does not see: -inf over their scores
                // in tensor memory.  This and the other seldom-run parts are rolled
                // loops: what is run once for an item is fetched from far away, at
                // about 100 cycles for 8 instructions.
                if (active && !__all_sync(0xffffffffu, lim >= 128)) {
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        if (__all_sync(0xffffffffu, lim >= c + 32)) continue;
                        uint32_t w[32];
                        tmem_ld32(tS + c, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i >= lim) w[i] = 0xFF800000u;
                        tmem_st32(tS + c, w);
                    }
                    tmem_wait_st();
                }
                uint32_t s[4][32];
                float mx0 = 0.f, mx1 = 0.f;
                if (active) {
                    tmem_ld64_max(tS, s[0], s[1], mx0);
                    tmem_ld64_max(tS + 64, s[2], s[3], mx1);
                    tmem_wait_ld();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_SFREE + X));
                float f = 1.f;
                bool rescale = false;
                if (active) {
                    const float mx = fmaxf(mx0, mx1);
                    const float mt = mx * p.sc;
                    const bool grow = mt > m + kLazy;      // also the first visible key: m = -inf
                    if (grow) {
                        f = ex2_approx(m - mt);
                        l *= f;
                        m = mt;
                    }
                    const float neg = m == -INFINITY ? 0.f : -m;
                    float la[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float x0, x1;
                            fma2_bc(x0, x1, __uint_as_float(s[a][i]), __uint_as_float(s[a][i + 1]), p.sc, neg);
                            x0 = ex2_approx(x0);
                            x1 = ex2_approx(x1);
                            add2(la[i & 2], la[(i & 2) + 1], x0, x1);
                            s[a][i / 2] = pack2(x0, x1);
                        }
                    l += (la[0] + la[1]) + (la[2] + la[3]);
                    rescale = !fresh && __any_sync(0xffffffffu, grow);
                }
                // This group's product before is done: it has read P, and O may be
                // rescaled.  Warps without rows wait too: an arrival for the next
                // product before this one was issued would be lost.
                if (units > 0 && !mbar_spin_warp(bar(L::B_PV + X), (units - 1) & 1, abort_flag)) {
                    if (lane == 0) fail(R_ROWS, t);
                    break;
                }
                tc_fence_after();
                if (active) {
                    if (rescale) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tO + c * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(tO + c * 32, o);
                        }
                    }
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = s[a][i];
                        tmem_st16(tP + a * 16, w);
                    }
                    tmem_wait_st();
                }
                ++units;
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
#pragma unroll 1
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4*>(vr + (c >> 3) * kBlk + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_P + X));
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
#pragma unroll 1
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
                    // 32 channels at a time.  They leave through shared memory (Q's
                    // place: its products are done), so that a store's lanes share
                    // lines; a warp stages its own 32 rows.
                    const bool whole = (flags & N_WHOLE) != 0;
                    const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
                    const int64_t row0 = (int64_t)nt.slot * M + (kSplit ? 0 : X * 128) + (warp & 3) * 32;
                    const int64_t at = whole ? o_at : (valid ? (row0 + lane) * D : -1);
                    if (valid && !whole) p.part_ml[row0 + lane] = make_float2(m, l);
                    uint8_t* stage = sgen + (kSplit ? L::OFF_STAGE : L::OFF_Q + X * L::kTile) + (warp & 3) * 4096;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + c * 32, o);
                        tmem_wait_ld();
                        if constexpr (kSplit) {
                            // a group without a tile, or without a visible key, adds nothing
                            // (its O may hold anything)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 y = *reinterpret_cast<const float4*>(jr + (((c * 8 + i) ^ (row & kSw)) << 4));
                                const float yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float z = __uint_as_float(o[4 * i + e]);
                                    o[4 * i + e] = __float_as_uint((fa == 0.f ? 0.f : z * fa) + (fb == 0.f ? 0.f : yy[e] * fb));
                                }
                            }
                        }
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = pack2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        }
                        if (whole) stage_out<4>(stage, o, at, p.o + c * 32, lane);
                        else stage_out<8>(stage, o, at, p.part_o + c * 32, lane);
                    }
                }
                tc_fence_before();
                ++items;
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    }
    if (warp == kWarpLoad) {
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
    } else if (warp == kWarpS || warp == kWarpPV) {
        // ===================================================== MMA issuers
        // Issuing takes about 48 cycles of a thread per instruction and 45 per
        // wait or commit: one thread for both products needs longer than the
        // 1,024 cycles that a unit's products take.  The two touch different
        // tensor memory, so each has a thread of its own.
        constexpr int kUnitsPerTile = kSplit ? 1 : 2;
        const int U = count * kUnitsPerTile;
        bool ok = true;
        int u = 0;
        if (warp == kWarpS) {
            constexpr uint32_t kIdescQK = idesc_bf16(128, false);
            const uint64_t dQ = sdesc_sw128(sbase + L::OFF_Q);
            const uint64_t dK = sdesc_sw128(sbase + L::OFF_K);
            int items = 0;
            for (; u < U; ++u) {
                const int t = u / kUnitsPerTile, st = t % NS, X = u & 1;
                if (u % kUnitsPerTile == 0) {
                    if (!mbar_spin_warp(bar(L::B_KF + st), (t / NS) & 1, abort_flag)) { ok = false; break; }
                    // a new item's Q: written when the item before is through
                    if (notes[t % kNotes].flags & N_FIRST) {
                        if (!mbar_spin_warp(bar(L::B_Q), items & 1, abort_flag)) { ok = false; break; }
                        ++items;
                    }
                }
                const int before = u - L::kSBufs;          // the unit that used the buffer last: its scores are in registers
                if (before >= 0 && !mbar_spin_warp(bar(L::B_SFREE + (before & 1)), (before >> 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t a = dQ + (uint64_t)((kSplit ? 0 : X * L::kTile) >> 4);
                const uint64_t b = dK + (uint64_t)((st * L::kTile) >> 4);
                const uint32_t d = tmem + (L::kSBufs == 2 ? 128u * X : 0u);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
                    mma_ss_elect(d, a + o, b + o, kIdescQK, kk > 0 ? 1u : 0u);
                }
                commit_elect(bar(L::B_S + X));
                if (u % kUnitsPerTile == kUnitsPerTile - 1) commit_elect(bar(L::B_KE + st));
            }
        } else {
            constexpr uint32_t kIdescPV = idesc_bf16(D, true);
            const uint64_t dV = sdesc_n_major(sbase + L::OFF_V);
            uint32_t summed = 0;                          // bit X: group X has a product in this item
            bool last = false;
            for (; u < U; ++u) {
                const int t = u / kUnitsPerTile, st = t % NS, X = u & 1;
                if (u % kUnitsPerTile == 0) {
                    if (!mbar_spin_warp(bar(L::B_VF + st), (t / NS) & 1, abort_flag)) { ok = false; break; }
                    const int f = notes[t % kNotes].flags;
                    if (f & N_FIRST) summed = 0;
                    last = (f & N_LAST) != 0;
                }
                if (!mbar_spin_warp(bar(L::B_P + X), (u >> 1) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint64_t b = dV + (uint64_t)((st * L::kTile) >> 4);
                const uint32_t dO = tmem + L::TM_O + (uint32_t)D * X, aP = tmem + L::TM_P + 64u * X;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ts_elect(dO, aP + kk * 8, b + (uint64_t)(kk * (2048 >> 4)), kIdescPV,
                               kk > 0 || ((summed >> X) & 1u) ? 1u : 0u);
                summed |= 1u << X;
                commit_elect(bar(L::B_PV + X));
                if (u % kUnitsPerTile == kUnitsPerTile - 1) {
                    commit_elect(bar(L::B_VE + st));
                    if (last) commit_elect(bar(L::B_ODONE));
                }
            }
        }
        if (!ok && lane == 0) fail(R_ISSUE, u);
        const int drain = L::B_DRAIN + (warp == kWarpS ? 0 : 1);
        commit_elect(bar(drain));                           // all products done before teardown
        const int zero = 0;
        mbar_wait_warp(bar(drain), 0, &zero);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpS) {
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
