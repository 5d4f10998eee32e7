// sage_paged_tiles.cu - attention over a page cache for many query rows, on
// the tcgen05 tensor cores.
//
// A persistent CTA is one worker of the list of sage_paged_sched.cuh with
// 128-key tiles.  Its query rows form groups of 128; a "unit" is one group's
// S = Q K^T and O += P V of one tile.
//   kGroups = 2 (items of 256 rows, one CTA per SM): both groups see every
//     tile and take turns at the tensor core, so that one group's softmax runs
//     beside the other's products and a K or V tile is loaded once for both.
//   kGroups = 1 (items of 128 rows, two CTAs per SM): a lone group's products
//     and softmax follow one another; the two CTAs of an SM overlap instead,
//     each with its own items, which also hides the ends of short items.
//
// Warp roles.  kGroups = 2: 384 threads, kGroups = 1: 192.
//   warps 0-3 (4-7)  softmax of group 0 (1), one thread per row: S from tensor
//                    memory, mask, online maximum and sum, P in BF16 back to
//                    tensor memory; the output from tensor memory
//   loader           the pages of a K and of a V tile by TMA through rings of
//                    stages; it alone walks the list and leaves a note for
//                    each tile
//   Q loader         the rows of the next item as soon as the last scores of
//                    this one are computed (kGroups = 1: the loader)
//   issuers          kGroups = 2: one thread for S = Q K^T and one for O += P V
//                    (issuing takes about 48 cycles of a thread per
//                    instruction and 45 per wait or commit, so one thread
//                    would need longer than the 1,024 cycles of a unit's
//                    products); kGroups = 1: one thread for both
//   kGroups = 2: the last four warps' registers go to the softmax (setmaxnreg:
//   2 x 128 x 224 + 128 x 56 = 384 x 168).
// Tensor memory, kGroups = 2: O of both groups in the top 2 D columns, P of
// each group beside its S.  D = 128: [S 128 | P0 64 | P1 64 | O0 | O1], one S
// for both groups: a group loads its scores into registers at once and frees
// it, so the next scores are computed while the exponentials run.  D = 64:
// [S0 128 | S1 128 | P0 | P1 | O0 | O1].  kGroups = 1: 256 columns; D = 128:
// [S 128, its first half P | O 128], D = 64: [S 128 | P 64 | O 64].
//
// The reference of the exponentials follows the row maximum lazily: O is
// rescaled only when the maximum has grown by more than 2^8 since the last
// rescale.  The weights then reach 2^8 at most, which BF16 holds at the same
// relative error, and the rescale (a round trip of O through registers)
// almost never runs.
//
// What runs once for an item is fetched from far away, at about 100 cycles for
// every 8 instructions, so the seldom-run parts are rolled loops.
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

constexpr int kNotes = 8;
constexpr int kItemNotes = 8;
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
// ... and about an item, to the Q loader.
struct ItemNote {
    int b, h, rt, n;
    int tile;                                             // its first tile in this worker
    int pad[3];
};
enum { N_FIRST = 1, N_LAST = 2, N_OWN = 4, N_WHOLE = 8 };  // of its item in this worker; own keys; item not shared

template <int D, int kGroups>
struct TilesShape {
    static constexpr int M = 128 * kGroups;
    static constexpr int kThreads = kGroups == 2 ? 384 : 192;
    static constexpr int kWarpLoad = 4 * kGroups, kWarpS = kWarpLoad + 1, kWarpPV = kGroups == 2 ? kWarpS + 1 : kWarpS;
    static constexpr int kWarpQ = kGroups == 2 ? kWarpPV + 1 : kWarpLoad;
    static constexpr int kCtasPerSm = kGroups == 2 ? 1 : 2;
    static constexpr int kNB = D / 64;                    // 64-channel blocks of a row
    static constexpr uint32_t kTile = kNB * kBlk;         // bytes of a K (or V) tile, and of a group's Q
    static constexpr int kNS = (D == 128 ? 1 : 2) * kGroups;       // K and V stages
    // tensor memory
    static constexpr uint32_t kCols = kGroups == 2 ? 512 : 256;
    static constexpr bool kAlias = D == 128 && kGroups == 1;       // P over its own S
    static constexpr int kSBufs = D == 128 ? 1 : kGroups;
    static constexpr uint32_t TM_P = kAlias ? 0 : 128 * kSBufs;    // + 64 X
    static constexpr uint32_t TM_O = kAlias ? 128 : TM_P + 64 * kGroups;   // + D X
    // shared memory
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = kGroups * kTile;
    static constexpr uint32_t OFF_V = OFF_K + kNS * kTile;
    static constexpr uint32_t OFF_STAGE = OFF_V + kNS * kTile;     // rows on their way out, 2 KB a warp
    static constexpr uint32_t OFF_BAR = OFF_STAGE + kGroups * 4 * 2048;
    static constexpr int B_Q = 0, B_ODONE = 1, B_DRAIN = 2;
    static constexpr int B_S = 4, B_SFREE = 6, B_P = 8, B_PV = 10;                // one of each per group
    static constexpr int B_KF = 12, B_KE = B_KF + kNS, B_VF = B_KE + kNS, B_VE = B_VF + kNS, B_NOTE = B_VE + kNS;
    static constexpr int B_ITEM = B_NOTE + kNotes;
    static constexpr int kBars = B_ITEM + kItemNotes;
    static constexpr uint32_t OFF_NOTE = OFF_BAR + (kBars * 8 + 15) / 16 * 16;
    static constexpr uint32_t OFF_ITEM = OFF_NOTE + kNotes * sizeof(TileNote);
    static constexpr uint32_t OFF_SCAN = OFF_ITEM + kItemNotes * sizeof(ItemNote);    // int [16], int2
    static constexpr uint32_t OFF_TMEM = OFF_SCAN + 80;
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

// Store 64 bytes of each lane's row (at base + at; at < 0: no row) through 32
// staged rows.  All 32 lanes call it together.
template <class T>
__device__ __forceinline__ void stage_out(uint8_t* stage, const uint32_t (&w)[16], int64_t at, T* base, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), c = lane & 3;
        const int64_t a = __shfl_sync(0xffffffffu, at, r);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
        if (a >= 0) reinterpret_cast<uint4*>(base + a)[c] = v;
    }
    __syncwarp();
}

template <int D, int kGroups>
__global__ void __launch_bounds__(TilesShape<D, kGroups>::kThreads, TilesShape<D, kGroups>::kCtasPerSm)
paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ PagedParams p) {
    using L = TilesShape<D, kGroups>;
    constexpr int M = L::M, NS = L::kNS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t sbase = (raw_base + 1023u) & ~1023u;
    uint8_t* sgen = smem_raw + (sbase - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_trigger();
    auto bar = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)i; };
    TileNote* notes = reinterpret_cast<TileNote*>(sgen + L::OFF_NOTE);
    ItemNote* item_notes = reinterpret_cast<ItemNote*>(sgen + L::OFF_ITEM);
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
        mbar_init(bar(L::B_Q), 1);
        mbar_init(bar(L::B_ODONE), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::B_DRAIN + i), 1);
            mbar_init(bar(L::B_S + i), 1);
            mbar_init(bar(L::B_SFREE + i), 4);            // one arrival a warp
            mbar_init(bar(L::B_P + i), 4);
            mbar_init(bar(L::B_PV + i), 1);
        }
        for (int i = 0; i < 4 * NS; ++i) mbar_init(bar(L::B_KF + i), 1);
        for (int i = 0; i < kNotes + kItemNotes; ++i) mbar_init(bar(L::B_NOTE + i), 1);
        fence_mbar_init();
    }
    if (warp == L::kWarpS) {
        tmem_alloc(sbase + L::OFF_TMEM, L::kCols);
        tmem_relinquish();
    }
    if (warp == L::kWarpLoad && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    tc_fence_before();
    const PagedSched<M, 128> sched(p);
    int* red = reinterpret_cast<int*>(sgen + L::OFF_SCAN);
    int2* found = reinterpret_cast<int2*>(sgen + L::OFF_SCAN + 64);
    const int worker = blockIdx.x;
    const int total = paged_scan<M, 128, L::kThreads, 1>(sched, worker, 0, found, red, false);   // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int per = sched.per_worker(total);
    const int t0 = min(worker * per, total);
    const int count = min(per, total - t0);               // tiles of this worker, perhaps none

    if (warp < 4 * kGroups) {
        // ===================================================== softmax
        if constexpr (kGroups == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int X = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + (L::kSBufs == 2 ? 128u * X : 0u);
        const uint32_t tP = tmem + lane_base + L::TM_P + 64u * X, tO = tmem + lane_base + L::TM_O + (uint32_t)D * X;
        float m = -INFINITY, l = 0.f;                     // reference of the exponentials (log2 domain), sum
        bool fresh = true;                                // no tile of this item yet: O holds nothing
        bool valid = false, active = false;               // this row exists; some row of this warp does
        int lim_own = 0;                                  // own keys this row sees
        int64_t o_at = -1;                                // offset of this row's output, -1: none
        int items = 0;
        for (int t = 0; t < count; ++t) {
            if (!mbar_spin_warp(bar(L::B_NOTE + t % kNotes), (t / kNotes) & 1, abort_flag)) {
                if (lane == 0) fail(R_ROWS, t);
                break;
            }
            const TileNote& nt = notes[t % kNotes];
            const int flags = nt.flags;
            if (flags & N_FIRST) {
                PagedPlace x{};
                x.b = nt.b; x.h = nt.h; x.rt = nt.rt; x.n = nt.n; x.len = nt.len;
                int rb, ri, rh;
                valid = paged_row(sched, x, X * 128 + row, rb, ri, rh);
                active = __any_sync(0xffffffffu, valid);
                lim_own = nt.len;
                if (p.causal && nt.b >= 0) lim_own = min(nt.len, nt.len - nt.n + ri + 1);
                o_at = valid ? rb * p.osb + rh * p.osh + ri * p.osn : -1;
                m = -INFINITY; l = 0.f; fresh = true;
            }
            const int nkeys = nt.nkeys;
            int lim = nkeys;                              // keys of the tile this row sees (may be negative)
            if (flags & N_OWN) lim = min(lim, lim_own - nt.key0);
            if (!mbar_spin_warp(bar(L::B_S + X), t & 1, abort_flag)) {
                if (lane == 0) fail(R_ROWS, t);
                break;
            }
            tc_fence_after();
            // keys that some row of this warp does not see: -inf over their scores
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
            if constexpr (!L::kAlias) {                   // (P over S: the next scores wait for its product)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_SFREE + X));
            }
            float f = 1.f;
            bool rescale = false;
            if (active) {
                const float mt = fmaxf(mx0, mx1) * p.sc;
                const bool grow = mt > m + kLazy;         // also the first visible key: m = -inf
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
            // rescaled.  (P over S: these scores were issued behind it.)  Warps
            // without rows wait too: an arrival for the next product before this
            // one was issued would be lost.
            if (!L::kAlias && t > 0 && !mbar_spin_warp(bar(L::B_PV + X), (t - 1) & 1, abort_flag)) {
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
            fresh = false;
            tc_fence_before();
            // V rows behind the last key: whatever they hold times a weight of 0
            // must be 0 (group 0's product is the first to read them)
            if (nkeys < 128 && X == 0) {
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
            if (flags & N_LAST) {
                const bool whole = (flags & N_WHOLE) != 0;
                const int64_t row0 = (int64_t)nt.slot * M + X * 128 + (warp & 3) * 32;
                if (!mbar_wait_warp(bar(L::B_ODONE), items & 1, abort_flag)) {
                    if (lane == 0) fail(R_ROWS, t);
                    break;
                }
                tc_fence_after();
                if (active) {
                    // 64 bytes of each row at a time leave through shared memory, so
                    // that a store's lanes share lines; a warp stages its own rows.
                    uint8_t* stage = sgen + L::OFF_STAGE + warp * 2048;
                    if (whole) {
                        const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32], w[16];
                            tmem_ld32(tO + c * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = pack2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                            stage_out(stage, w, o_at, p.o + c * 32, lane);
                        }
                    } else {
                        if (valid) p.part_ml[row0 + lane] = make_float2(m, l);
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tO + c * 16, o);
                            tmem_wait_ld();
                            stage_out(stage, o, valid ? (row0 + lane) * D : -1, p.part_o + c * 16, lane);
                        }
                    }
                }
                tc_fence_before();
                ++items;
            }
        }
    } else if constexpr (kGroups == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    }
    // Fetch an item's Q rows by 16-byte copies,
    // neighbouring lanes on neighbouring chunks of a row, into the K-major 128-byte
    // swizzle.  Its place is free once the scores of the tile before are computed,
    // which is well before that item's output is written.  One warp.
    auto load_q = [&](const ItemNote& nt) -> bool {
        const int t = nt.tile;
        PagedPlace x{};
        x.b = nt.b; x.h = nt.h; x.rt = nt.rt; x.n = nt.n;
        if (t > 0 && !mbar_wait_warp(bar(L::B_KE + (t - 1) % NS), ((t - 1) / NS) & 1, abort_flag)) return false;
        constexpr int kC = D / 8, kR = 32 / kC;           // 16-byte chunks of a row, rows a copy covers
#pragma unroll 1
        for (int r0 = 0; r0 < M; r0 += 32) {
            int rb, ri, rh;
            const bool in = paged_row(sched, x, r0 + lane, rb, ri, rh);
            const int64_t q_at = in ? rb * p.qsb + rh * p.qsh + ri * p.qsn : -1;
#pragma unroll 4
            for (int i = 0; i < kC; ++i) {
                const int r = r0 + i * kR + lane / kC, c = lane % kC;
                const int64_t at = __shfl_sync(0xffffffffu, q_at, i * kR + lane / kC);
                cp_async16(sbase + L::OFF_Q + (r >> 7) * L::kTile + (c >> 3) * kBlk + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4),
                           at >= 0 ? p.q + at + c * 8 : p.q, at >= 0 ? 16u : 0u);
            }
        }
        return true;
    };
    auto q_ready = [&]() {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_Q));
    };
    if (kGroups == 2 && warp == L::kWarpQ) {
        // ===================================================== Q loader
        // Slots of notes are not overrun: item k + 8 begins 8 tiles or more behind
        // item k, and the loader is at most its stages ahead of the scores.
        for (int k = 0;; ++k) {
            const ItemNote& nt = item_notes[k % kItemNotes];
            if (!mbar_wait_warp(bar(L::B_ITEM + k % kItemNotes), (k / kItemNotes) & 1, abort_flag)) {
                if (lane == 0) fail(R_LOAD, -1);
                break;
            }
            if (nt.tile >= count) break;                  // no more items
            if (!load_q(nt)) {
                if (lane == 0) fail(R_LOAD, nt.tile);
                break;
            }
            q_ready();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == L::kWarpLoad) {
        // ===================================================== TMA producer
        // Whether this worker's run opens inside an item and is the first to do
        // so: then the item is joined from its parts afterwards.
        int4 cut = make_int4(-1, 0, 0, 0);                // request, key head, row tile, parts
        PagedPlace at{};
        if (count > 0) {
            at = paged_place(sched, found[0], t0);
            if (p.cuts != nullptr && at.tile > 0) {
                const int start = t0 - at.tile, w0 = start / per;
                if (w0 == worker - 1) cut = make_int4(at.b, at.h, at.rt, (start + at.ntiles - 1) / per - w0 + 1);
            }
        }
        if (p.cuts != nullptr && lane == 0) p.cuts[worker] = cut;
        const int per_tile = 128 >> p.page_shift;         // pages of a whole tile
        auto page_of = [&](const PagedSpan& sp, const PagedPlace& x) -> int {
            if (lane >= per_tile || (lane << p.page_shift) >= sp.nkeys) return 0;
            const int j = (sp.key0 >> p.page_shift) + lane;
            return sp.own ? __ldg(p.table + (int64_t)x.b * p.table_stride + j) : __ldg(p.ptable + j);
        };
        PagedSpan span{};
        int page = 0;
        if (count > 0) {
            span = paged_span(sched, at);
            page = page_of(span, at);
        }
        bool first = true;
        int run0 = at.tile;                               // the item's first tile in this worker
        int loaded_k = 0, loaded_v = 0;                   // tiles whose copies were issued
        int items = 0;                                    // items noted
        auto post_item = [&](int t) {                     // lane 0
            ItemNote& in = item_notes[items % kItemNotes];
            in.b = at.b; in.h = at.h; in.rt = at.rt; in.n = at.n; in.tile = t;
            if (kGroups == 2) mbar_arrive(bar(L::B_ITEM + items % kItemNotes));
        };
        bool ok = true;
#pragma unroll 1
        for (int t = 0; t < count; ++t) {
            const int st = t % NS, ph = (t / NS) & 1;
            const bool mine = lane < per_tile && (lane << p.page_shift) < span.nkeys;
            const uint32_t bytes = (uint32_t)((span.nkeys + p.page - 1) >> p.page_shift) * (uint32_t)(p.page * 128 * L::kNB);
            const uint32_t off = (uint32_t)(lane * p.page) * 128u;
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
                if (first) post_item(t);
                mbar_arrive(bar(L::B_NOTE + t % kNotes));
                mbar_arrive_expect_tx(bar(L::B_KF + st), bytes);
            }
            if (first) ++items;
            __syncwarp();
            // a page outside the cache: the copy reads zeros there
            if (mine && (unsigned)page >= (unsigned)p.num_pages && atomicCAS(p.status, 0, kErrPage) == 0) p.status[3] = page;
            if (mine) {
#pragma unroll
                for (int hb = 0; hb < L::kNB; ++hb)
                    tma_load_4d(sbase + L::OFF_K + st * L::kTile + hb * kBlk + off, &tm_k, hb * 64, 0, at.h, page,
                                bar(L::B_KF + st));
            }
            loaded_k = t + 1;
            if (kGroups == 1 && first && !load_q(item_notes[(items - 1) % kItemNotes])) { ok = false; break; }
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
            if (kGroups == 1 && first) q_ready();
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
        // (its slot is free for the same reason)
        if (kGroups == 2 && ok && lane == 0) post_item(count);
        asm volatile("cp.async.wait_all;" ::: "memory");
        // every copy issued lands before the CTA may exit
        const int zero = 0;
        for (int i = 0; i < NS; ++i) {
            const int tk = loaded_k - 1 - i, tv = loaded_v - 1 - i;
            if (tk >= 0) mbar_wait_warp(bar(L::B_KF + tk % NS), (tk / NS) & 1, &zero);
            if (tv >= 0 && p.fault_mode != 1) mbar_wait_warp(bar(L::B_VF + tv % NS), (tv / NS) & 1, &zero);
        }
    } else if (warp == L::kWarpS || warp == L::kWarpPV) {
        // ===================================================== MMA issuers
        constexpr uint32_t kIdescQK = idesc_bf16(128, false);
        constexpr uint32_t kIdescPV = idesc_bf16(D, true);
        const uint64_t dQ = sdesc_sw128(sbase + L::OFF_Q);
        const uint64_t dK = sdesc_sw128(sbase + L::OFF_K);
        const uint64_t dV = sdesc_n_major(sbase + L::OFF_V);
        const int U = count * kGroups;
        int items = 0;                                    // items opened
        uint32_t summed = 0;                              // bit X: group X has a product in this item
        bool last = false;                                // the tile is its item's last
        auto issue_s = [&](int u) -> bool {
            const int t = u / kGroups, st = t % NS, X = u % kGroups;
            if (X == 0) {
                if (!mbar_spin_warp(bar(L::B_KF + st), (t / NS) & 1, abort_flag)) return false;
                // a new item's Q
                if (notes[t % kNotes].flags & N_FIRST) {
                    if (!mbar_spin_warp(bar(L::B_Q), items & 1, abort_flag)) return false;
                    ++items;
                }
            }
            if constexpr (!L::kAlias) {                   // the unit that used the buffer last has its scores in registers
                const int before = u - L::kSBufs;
                if (before >= 0 && !mbar_spin_warp(bar(L::B_SFREE + before % kGroups), (before / kGroups) & 1, abort_flag))
                    return false;
            }
            tc_fence_after();
            const uint64_t a = dQ + (uint64_t)((X * L::kTile) >> 4);
            const uint64_t b = dK + (uint64_t)((st * L::kTile) >> 4);
            const uint32_t d = tmem + (L::kSBufs == 2 ? 128u * X : 0u);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
                mma_ss_elect(d, a + o, b + o, kIdescQK, kk > 0 ? 1u : 0u);
            }
            commit_elect(bar(L::B_S + X));
            if (X == kGroups - 1) commit_elect(bar(L::B_KE + st));
            return true;
        };
        auto issue_pv = [&](int u) -> bool {
            const int t = u / kGroups, st = t % NS, X = u % kGroups;
            if (X == 0) {
                if (!mbar_spin_warp(bar(L::B_VF + st), (t / NS) & 1, abort_flag)) return false;
                const int f = notes[t % kNotes].flags;
                if (f & N_FIRST) summed = 0;
                last = (f & N_LAST) != 0;
            }
            if (!mbar_spin_warp(bar(L::B_P + X), t & 1, abort_flag)) return false;
            tc_fence_after();
            const uint64_t b = dV + (uint64_t)((st * L::kTile) >> 4);
            const uint32_t dO = tmem + L::TM_O + (uint32_t)D * X, aP = tmem + L::TM_P + 64u * X;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_ts_elect(dO, aP + kk * 8, b + (uint64_t)(kk * (2048 >> 4)), kIdescPV,
                             kk > 0 || ((summed >> X) & 1u) ? 1u : 0u);
            summed |= 1u << X;
            if constexpr (!L::kAlias) commit_elect(bar(L::B_PV + X));
            if (X == kGroups - 1) {
                commit_elect(bar(L::B_VE + st));
                if (last) commit_elect(bar(L::B_ODONE));
            }
            return true;
        };
        bool ok = true;
        int u = 0;
        if constexpr (kGroups == 2) {
            if (warp == L::kWarpS) {
                for (; u < U && ok; ++u) ok = issue_s(u);
            } else {
                for (; u < U && ok; ++u) ok = issue_pv(u);
            }
        } else {
            for (; u < U && ok; ++u) ok = issue_s(u) && issue_pv(u);
        }
        if (!ok && lane == 0) fail(R_ISSUE, u);
        const int drain = L::B_DRAIN + (warp == L::kWarpS ? 0 : 1);
        commit_elect(bar(drain));                         // all products done before teardown
        const int zero = 0;
        mbar_wait_warp(bar(drain), 0, &zero);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == L::kWarpS) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
}

// ---------------------------------------------------------------------------
// Join the items that a worker boundary cuts (list without shared prefix
// items; whole items were written by the kernel above).  blockIdx.x + 1 is
// the worker behind the boundary, blockIdx.y a group of 32 rows.
// ---------------------------------------------------------------------------
template <int D, int M>
__global__ void __launch_bounds__(256) paged_cuts_kernel(const __grid_constant__ PagedParams p) {
    constexpr int V = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.x + 1;
    pdl_wait();
    const int4 cut = __ldcg(p.cuts + w);
    if (cut.x < 0) return;
    const PagedSched<M, 128> s(p);
    PagedPlace x{};
    x.b = cut.x; x.h = cut.y; x.rt = cut.z;
    x.n = s.q_rows(x.b);
    const int r0 = (int)blockIdx.y * 32 + warp * 4;        // four rows of this warp
    if ((x.rt * M + r0) / p.G >= x.n) return;
    float acc[4][V], m[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = -INFINITY;
        l[k] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[k][v] = 0.f;
    }
#pragma unroll 1
    for (int j = 0; j < cut.w; ++j) {                      // part 0: the second slot of worker w - 1
        const int64_t q = (int64_t)(j == 0 ? 2 * (w - 1) + 1 : 2 * (w - 1 + j)) * M + r0;
        float2 ml[4];
        float y[4][V];
#pragma unroll
        for (int k = 0; k < 4; ++k) {                      // rows that do not exist hold anything and are not stored
            ml[k] = __ldcg(p.part_ml + q + k);
#pragma unroll
            for (int v = 0; v < V; ++v) y[k][v] = __ldcg(p.part_o + (q + k) * D + lane + 32 * v);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float mn = fmaxf(m[k], ml[k].x);
            const float ms = mn == -INFINITY ? 0.f : mn;
            const float fa = ex2_approx(m[k] - ms), fb = ex2_approx(ml[k].x - ms);
            l[k] = l[k] * fa + ml[k].y * fb;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[k][v] = acc[k][v] * fa + y[k][v] * fb;
            m[k] = mn;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        int b, i, hq;
        if (!paged_row(s, x, r0 + k, b, i, hq)) continue;
        const float inv = l[k] == 0.f ? 0.f : __fdiv_rn(1.f, l[k]);
        uint16_t* dst = p.o + b * p.osb + hq * p.osh + (int64_t)i * p.osn + lane;
#pragma unroll
        for (int v = 0; v < V; ++v) dst[32 * v] = (uint16_t)pack2(acc[k][v] * inv, 0.f);
    }
}

template <int D, int kGroups>
cudaError_t launch_one(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    using L = TilesShape<D, kGroups>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(paged_tiles_kernel<D, kGroups>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    paged_tiles_kernel<D, kGroups><<<p.workers, L::kThreads, L::kSmem, s>>>(tk, tv, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.pre_rt == 0 && p.workers > 1)
        e = launch_after(paged_cuts_kernel<D, L::M>, dim3((unsigned)p.workers - 1, L::M / 32), dim3(256), 0, s, true, p);
    return e;
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedParams& p, int D, int groups, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
    if (D == 64) return groups == 1 ? launch_one<64, 1>(p, tk, tv, s) : launch_one<64, 2>(p, tk, tv, s);
    return groups == 1 ? launch_one<128, 1>(p, tk, tv, s) : launch_one<128, 2>(p, tk, tv, s);
}

}  // namespace sage
