// sage_paged_tiles.cu - attention over a page cache for many query rows, on
// the tcgen05 tensor cores.
//
// A persistent CTA is one worker of the list of sage_paged_sched.cuh with
// 128-key tiles, or it takes one item of that list whole.  Its query rows form groups of 128; a "unit" is one group's
// S = Q K^T and O += P V of one tile.
//   kGroups = 2 (one CTA per SM): both groups see every tile and take turns at
//     the tensor core, so that one group's softmax runs beside the other's
//     products and a K or V tile is loaded once for both.
//   kGroups = 1 (two CTAs per SM): items of one group; the two CTAs of an SM
//     overlap instead, each with its own items, which hides the ends of short
//     items.
//
// Warps (a group's are numbered after one another):
//   8 a group  softmax.  A row belongs to two threads, in warps that see the
//              same quarter of tensor memory: "half" 0 owns keys 0-63 of every
//              tile and the lower half of the channels, half 1 the others.
//              They exchange their maxima through shared memory.  Two halves
//              keep twice the warps per scheduler that one thread a row would,
//              which is what hides the latency of their chain of tensor-memory
//              load, exponentials and store.
//   loader     the rows of an item and the pages of its K and V tiles by TMA;
//              it alone walks the list and leaves a note for each item
//   issuers    kGroups = 2: one thread for S and one for PV (an instruction
//              takes about 48 cycles of the issuing thread, a wait or commit
//              45: one thread, in the order S(u), PV(u - 2), takes 209 us where
//              the two take 179); kGroups = 1: one thread for both
//   kGroups = 2 has one more warp, idle: it completes the four whose registers
//   go to the softmax (setmaxnreg: 512 x 104 + 128 x 56 <= 640 x 96).
// Tensor memory: [S 128 | P 64 a group | O D a group].  Both groups share S: a
// group loads its scores into registers at once and frees it, so the next
// scores are computed while the exponentials run, and the two groups fall into
// turns by themselves.  (Each group's P over its own S, every unit a chain S,
// softmax, PV: the groups fall into step and leave the tensor core idle
// meanwhile, 2,250 cycles a unit.  An S for each group, at D = 64 and with
// prompts from the list: 46.6 us where the shared one took 44.3.)  One group of D = 128, with 256 columns:
// [S 128, its first half P | O 128].
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

constexpr int kItemNotes = 16;
constexpr float kLazy = 8.f;                              // log2 of the weights' bound
constexpr uint32_t kBlk = 128 * 128;                      // 128 rows x 64 channels

enum TileRole { R_ROWS = 6, R_LOAD = 7, R_ISSUE = 8 };

// What the loader says about an item.
struct ItemNote {
    int b, h, rt;
    int n, len;                                           // the request's query tokens and own keys
    int tile, run;                                        // its first tile in this worker, and how many (0: no item)
    int slot;                                             // of a partial result (of the prefix's, or the others')
    int whole;                                            // no other worker shares it: the output is final
    int pad[3];
};

template <int D, int kGroups>
struct TilesShape {
    static constexpr int M = 128 * kGroups;
    static constexpr int kWarpLoad = 8 * kGroups, kWarpIssue = kWarpLoad + 1;     // + X
    static constexpr int kThreads = kGroups == 2 ? 640 : 320;
    static constexpr int kCtasPerSm = kGroups == 2 ? 1 : 2;
    static constexpr int kNB = D / 64;                    // 64-channel blocks of a row
    static constexpr uint32_t kTile = kNB * kBlk;         // bytes of a K (or V) tile, and of a group's Q
    static constexpr int kNS = (D == 128 ? 1 : 2) * kGroups;       // K and V stages
    static constexpr uint32_t kCols = 256 * kGroups;      // tensor memory
    static constexpr bool kAlias = D == 128 && kGroups == 1;       // P over its S
    static constexpr uint32_t TM_P = kAlias ? 0 : 128;             // + 64 X
    static constexpr uint32_t TM_O = kAlias ? 128 : TM_P + 64 * kGroups;           // + D X
    // shared memory
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = kGroups * kTile;
    static constexpr uint32_t OFF_V = OFF_K + kNS * kTile;
    static constexpr uint32_t OFF_STAGE = OFF_V + kNS * kTile;     // rows on their way out, 1 KB a warp
    static constexpr uint32_t OFF_XM = OFF_STAGE + kGroups * 8 * 1024;            // float [2 turns][group][half][128]
    static constexpr uint32_t OFF_BAR = OFF_XM + kGroups * 2048;
    static constexpr int B_Q = 0, B_DRAIN = 1;            // B_DRAIN: + X
    static constexpr int B_S = 3, B_P = 5, B_ODONE = 7;   // + X
    static constexpr int B_X = 9;                         // + 4 X + quarter: the two halves of 32 rows
    static constexpr int B_SFREE = 17, B_PV = 19;         // + X (not kAlias)
    static constexpr int B_KF = 21, B_KE = B_KF + kNS, B_VF = B_KE + kNS, B_VE = B_VF + kNS, B_ITEM = B_VE + kNS;
    static constexpr int kBars = B_ITEM + kItemNotes;
    static constexpr uint32_t OFF_ITEM = OFF_BAR + (kBars * 8 + 15) / 16 * 16;
    static constexpr uint32_t OFF_SCAN = OFF_ITEM + kItemNotes * sizeof(ItemNote);   // int [20], int2
    static constexpr uint32_t OFF_TMEM = OFF_SCAN + 96;
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
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Store 32 bytes of each lane's row (at base + at; at < 0: no row) through 32
// staged rows, so that two lanes share a row's sector.  All 32 lanes call it.
template <class T>
__device__ __forceinline__ void stage_out(uint8_t* stage, const uint32_t (&w)[8], int64_t at, T* base, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4*>(stage + lane * 32 + ((i ^ ((lane >> 2) & 1)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = i * 16 + (lane >> 1), c = lane & 1;
        const int64_t a = __shfl_sync(0xffffffffu, at, r);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
        if (a >= 0) reinterpret_cast<uint4*>(base + a)[c] = v;
    }
    __syncwarp();
}

// What the kernel's work is: the list of the requests' own items, the list with
// the prefix's items in front, or an item for each CTA.
enum TileForm { F_LIST, F_PREFIX, F_ITEM };

template <int D, int kGroups, int kForm>
__global__ void __launch_bounds__(TilesShape<D, kGroups>::kThreads, TilesShape<D, kGroups>::kCtasPerSm)
paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qp,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ PagedParams p) {
    using L = TilesShape<D, kGroups>;
    constexpr int M = L::M, NS = L::kNS;
    constexpr bool kPre = kForm == F_PREFIX, kItem = kForm == F_ITEM;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t sbase = (raw_base + 1023u) & ~1023u;
    uint8_t* sgen = smem_raw + (sbase - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    auto bar = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)i; };
    ItemNote* notes = reinterpret_cast<ItemNote*>(sgen + L::OFF_ITEM);
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::B_DRAIN + i), 1);
            mbar_init(bar(L::B_S + i), 1);
            mbar_init(bar(L::B_P + i), 8);                // one arrival a warp
            mbar_init(bar(L::B_ODONE + i), 1);
            mbar_init(bar(L::B_SFREE + i), 8);
            mbar_init(bar(L::B_PV + i), 1);
        }
        for (int i = 0; i < 8; ++i) mbar_init(bar(L::B_X + i), 2);
        for (int i = L::B_KF; i < L::kBars; ++i) mbar_init(bar(i), 1);
        fence_mbar_init();
    }
    if (warp == L::kWarpLoad && lane == 0) {
        tma_prefetch_desc(kPre ? &tm_qp : &tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    pdl_wait();
    pdl_trigger();
    // Not before the wait: a kernel of another library that has let this one
    // start may still have to allocate its own.
    if (warp == L::kWarpIssue) {
        tmem_alloc(sbase + L::OFF_TMEM, L::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    const PagedSched<M, 128, kPre> sched(p);
    int* red = reinterpret_cast<int*>(sgen + L::OFF_SCAN);
    int2* found = reinterpret_cast<int2*>(sgen + L::OFF_SCAN + 80);
    const int worker = blockIdx.x;
    int t0 = 0, t1 = 0, per = 1;                          // this worker's run of the list
    if constexpr (kItem) {
        __syncthreads();                                  // a CTA takes an item
    } else {
        const int total = paged_scan<M, 128, kPre, L::kThreads, 1>(sched, worker, 0, found, red,      // ends with a barrier
                                                                   kPre && worker == 0 && p.start != nullptr);
        per = sched.share(total, p.workers, 0);
        t0 = min(worker * per, total);
        t1 = min(t0 + per, total);
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 8 * kGroups) {
        // ===================================================== softmax
        if constexpr (kGroups == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int X = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_base + 64u * half;
        const uint32_t tP = tmem + lane_base + L::TM_P + 64u * X + 32u * half;
        const uint32_t tO = tmem + lane_base + L::TM_O + (uint32_t)D * X + (uint32_t)half * (D / 2);
        const uint32_t bx = bar(L::B_X + 4 * X + quarter);
        // this row's place in the exchange, and its other half's
        float* xm = reinterpret_cast<float*>(sgen + L::OFF_XM) + (X * 2 + half) * 128 + row;
        const int other = half ? -128 : 128;
        constexpr int kTurn = kGroups * 256;
        int turn = 0;                                     // exchanges so far
        int t = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!mbar_wait_warp(bar(L::B_ITEM + k % kItemNotes), (k / kItemNotes) & 1, abort_flag)) {
                if (lane == 0) fail(R_ROWS, t);
                break;
            }
            const ItemNote& nt = notes[k % kItemNotes];
            if (nt.run == 0) break;
            const int ib = nt.b, len = nt.len, end = t + nt.run;
            int lim_own, rb, ri, rh;
            const bool valid = paged_row(sched, ib, nt.h, nt.rt, nt.n, X * 128 + row, rb, ri, rh);
            const bool active = __any_sync(0xffffffffu, valid);        // some row of this warp exists
            lim_own = p.causal && !(kPre && ib < 0) ? min(len, len - nt.n + ri + 1) : len;   // own keys this row sees
            float m = -INFINITY, l = 0.f;                 // reference of the exponentials (log2 domain), sum of this half
            bool fresh = true;                            // no tile of this item yet: O holds nothing
            int tile = nt.tile;
#pragma unroll 1
            for (; t < end; ++t, ++tile) {
                const PagedSpan span = paged_span(sched, ib, len, tile);
                // keys of this half that this row sees (may be negative)
                const int lim = (span.own ? min(span.nkeys, lim_own - span.key0) : span.nkeys) - half * 64;
                if (!mbar_wait_warp(bar(L::B_S + X), t & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                uint32_t s[2][32];
                float mx = 0.f;
                if (active) {
                    tmem_ld64_max(tS, s[0], s[1], mx);
                    tmem_wait_ld();
                }
                tc_fence_before();
                __syncwarp();
                if (!L::kAlias && lane == 0) mbar_arrive(bar(L::B_SFREE + X));
                float f = 1.f;
                bool rescale = false;
                if (active) {
                    if (!__all_sync(0xffffffffu, lim >= 64)) {
                        mx = -INFINITY;
#pragma unroll
                        for (int a = 0; a < 2; ++a)
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (a * 32 + i >= lim) s[a][i] = 0xFF800000u;      // -inf
                                mx = fmaxf(mx, __uint_as_float(s[a][i]));
                            }
                    }
                    float* at = xm + (turn & 1) * kTurn;
                    *at = mx;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bx);
                    if (!mbar_wait_warp(bx, turn & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();                     // the other half has its scores: P may lie over S
                    ++turn;
                    const float mt = fmaxf(mx, at[other]) * p.sc;
                    const bool grow = mt > m + kLazy;     // also the first visible key: m = -inf
                    if (grow) {
                        f = ex2_approx(m - mt);
                        l *= f;
                        m = mt;
                    }
                    rescale = !fresh && __any_sync(0xffffffffu, grow);
                    const float neg = m == -INFINITY ? 0.f : -m;
                    float la[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int a = 0; a < 2; ++a)
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
                }
                // This group's product before is done: it has read P, and O may be
                // rescaled.  (P over S: these scores were issued behind it.)  Warps
                // without rows wait too: an arrival for the next product before
                // this one was issued would be lost.
                if (!L::kAlias && t > 0 && !mbar_wait_warp(bar(L::B_PV + X), (t - 1) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                if (active) {
                    if (rescale) {
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(tO + c, o);
                        }
                    }
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
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
                if (span.nkeys < 128 && half == 0 && X == 0) {
                    if (!mbar_wait_warp(bar(L::B_VF + t % NS), (t / NS) & 1, abort_flag)) { ok = false; break; }
                    if (row >= span.nkeys) {
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
            if (!ok) break;
            // the item's end: the halves' sums together, the output from tensor memory
            float* at = xm + (turn & 1) * kTurn;
            if (active) {
                *at = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(bx);
            }
            if (!mbar_wait_warp(bar(L::B_ODONE + X), k & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            if (active) {
                if (!mbar_wait_warp(bx, turn & 1, abort_flag)) { ok = false; break; }
                ++turn;
                l += at[other];
                uint8_t* stage = sgen + L::OFF_STAGE + warp * 1024;
                if (kItem || (!kPre && nt.whole)) {
                    const int64_t o_at = valid ? rb * p.osb + rh * p.osh + ri * p.osn + half * (D / 2) : -1;
                    const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
#pragma unroll 1
                    for (int c = 0; c < D / 2; c += 16) {
                        uint32_t o[16], w[8];
                        tmem_ld16(tO + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = pack2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        if (o_at >= 0) {                  // a whole sector of its row: no staging needed
                            uint4* dst = reinterpret_cast<uint4*>(p.o + o_at + c);
                            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                        __syncwarp();
                    }
                } else {
                    const bool pre = kPre && ib < 0;
                    const int64_t part = (int64_t)nt.slot * (pre ? M : p.part_m) + X * 128 + row;
                    if (valid && half == 0) (pre ? p.pre_ml : p.part_ml)[part] = make_float2(m, l);
                    float* po = pre ? p.pre_o : p.part_o;
                    const int64_t part_at = valid ? part * D + half * (D / 2) : -1;
#pragma unroll 1
                    for (int c = 0; c < D / 2; c += 8) {
                        uint32_t o[8];
                        tmem_ld8(tO + c, o);
                        tmem_wait_ld();
                        stage_out(stage, o, part_at, po + c, lane);
                    }
                }
            }
            tc_fence_before();
        }
        if (!ok && lane == 0) fail(R_ROWS, t);
    } else if constexpr (kGroups == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    }
    if (warp == L::kWarpLoad) {
        // ===================================================== TMA producer
        // Whether this worker's run opens inside an item and is the first to do
        // so: then the item is joined from its parts afterwards.
        PagedCut cut{};
        cut.b = -1;
        PagedPlace at{};
        at.pos = t1;
        if constexpr (kItem) {
            // last row sets first: with a causal mask they are the longest
            const int each = p.B * p.Hkv, set = worker / each, rest = worker - set * each;
            at.rt = p.rt - 1 - set;
            at.b = rest / p.Hkv;
            at.h = rest - at.b * p.Hkv;
            at.n = sched.q_rows(at.b);
            at.len = sched.own_keys(at.b);
            t1 = at.ntiles = sched.item_tiles(at.n, at.len, at.rt);
        }
        else if (t0 < t1) at = paged_place(sched, found[0], t0);
        if (kForm == F_LIST && at.pos < t1 && at.tile > 0) {
            const int start = at.pos - at.tile, w0 = start / per;
            if (w0 == worker - 1) cut = PagedCut{at.b, at.h, at.rt, at.n, (start + at.ntiles - 1) / per - w0 + 1, {}};
        }
        if (kForm == F_LIST && lane == 0) p.cuts[worker] = cut;
        const int per_tile = 128 >> p.page_shift;         // pages of a whole tile
        PagedSpan span{};
        int page = 0;
        // this lane's page of the tile that `at` names
        auto look_up = [&]() {
            span = paged_span(sched, at.b, at.len, at.tile);
            page = 0;
            if (lane < per_tile && (lane << p.page_shift) < span.nkeys) {
                const int j = (span.key0 >> p.page_shift) + lane;
                page = span.own ? p.table[(int64_t)at.b * p.table_stride + j] : p.ptable[j];
            }
        };
        if (at.pos < t1) look_up();
        bool first = true;
        int items = 0;                                    // items noted
        int loaded_k = 0, loaded_v = 0;                   // tiles whose copies were issued
        bool ok = true;
#pragma unroll 1
        for (int t = 0; at.pos < t1; ++t) {
            const int st = t % NS, ph = (t / NS) & 1;
            const bool mine = lane < per_tile && (lane << p.page_shift) < span.nkeys;
            const uint32_t bytes = (uint32_t)((span.nkeys + p.page - 1) >> p.page_shift) * (uint32_t)(p.page * 128 * L::kNB);
            const uint32_t off = (uint32_t)(lane * p.page) * 128u;
            if (t >= NS && !mbar_wait_warp(bar(L::B_KE + st), ph ^ 1, abort_flag)) { ok = false; break; }
            if (lane == 0) {
                if (first) {
                    // Slots of notes are not overrun: item k + 16 begins 16 tiles or more
                    // behind item k, and the stages keep the loader that close.
                    ItemNote& nt = notes[items % kItemNotes];
                    nt.b = at.b; nt.h = at.h; nt.rt = at.rt;
                    nt.n = at.n; nt.len = at.len;
                    nt.tile = at.tile; nt.run = min(at.ntiles - at.tile, t1 - at.pos);
                    nt.slot = kPre ? worker + at.item : 2 * worker + (at.tile == 0 ? 1 : 0);
                    nt.whole = nt.run == at.ntiles;
                    mbar_arrive(bar(L::B_ITEM + items % kItemNotes));
                }
                mbar_arrive_expect_tx(bar(L::B_KF + st), bytes);
            }
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
            if (first) {
                // The item's rows: their place is free once the scores of the tile
                // before are computed, well before that item's output is written.
                if (t > 0 && !mbar_wait_warp(bar(L::B_KE + (t - 1) % NS), ((t - 1) / NS) & 1, abort_flag)) { ok = false; break; }
                if (lane == 0) {
                    const bool pre = kPre && at.b < 0;
                    const int tok = pre ? p.pre_tok : p.tok;
                    mbar_arrive_expect_tx(bar(L::B_Q), (uint32_t)(kGroups * L::kNB * tok * (pre ? p.pre_unit : p.G)) * 128u);
#pragma unroll
                    for (int X = 0; X < kGroups; ++X)
#pragma unroll
                        for (int hb = 0; hb < L::kNB; ++hb) {
                            const int g = (at.rt * kGroups + X) * tok;
                            tma_load_4d(sbase + L::OFF_Q + X * L::kTile + hb * kBlk, pre ? &tm_qp : &tm_q, hb * 64,
                                        at.h * p.G, pre ? 0 : g, pre ? g : at.b, bar(L::B_Q));
                        }
                }
                ++items;
            }
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
            if constexpr (kItem) ++at.pos, ++at.tile;
            else paged_next(sched, at);
            first = at.tile == 0;
            if (at.pos < t1) look_up();
        }
        if (!ok && lane == 0) fail(R_LOAD, loaded_v);
        if (ok && lane == 0) {                            // no more items
            notes[items % kItemNotes].run = 0;
            mbar_arrive(bar(L::B_ITEM + items % kItemNotes));
        }
        __syncwarp();
        // every copy issued lands before the CTA may exit
        const int zero = 0;
        if (items > 0) mbar_wait_warp(bar(L::B_Q), (items - 1) & 1, &zero);
        for (int i = 0; i < NS; ++i) {
            const int tk = loaded_k - 1 - i, tv = loaded_v - 1 - i;
            if (tk >= 0) mbar_wait_warp(bar(L::B_KF + tk % NS), (tk / NS) & 1, &zero);
            if (tv >= 0 && p.fault_mode != 1) mbar_wait_warp(bar(L::B_VF + tv % NS), (tv / NS) & 1, &zero);
        }
    } else if (warp >= L::kWarpIssue && warp < L::kWarpIssue + kGroups) {
        // ===================================================== MMA issuers
        constexpr uint32_t kIdescQK = idesc_bf16(128, false);
        constexpr uint32_t kIdescPV = idesc_bf16(D, true);
        const uint64_t dQ = sdesc_sw128(sbase + L::OFF_Q);
        const uint64_t dK = sdesc_sw128(sbase + L::OFF_K);
        const uint64_t dV = sdesc_n_major(sbase + L::OFF_V);
        // an item's first tile and the one behind its last, as S and as PV see them
        int s_items = 0, s_end = 0, v_items = 0, v_first = 0, v_end = 0;
        bool s_done = false, v_done = false;              // no more items
        auto issue_s = [&](int t) -> bool {
            if (t == s_end) {
                if (!mbar_wait_warp(bar(L::B_ITEM + s_items % kItemNotes), (s_items / kItemNotes) & 1, abort_flag)) return false;
                s_end = t + notes[s_items % kItemNotes].run;
                if (s_end == t) { s_done = true; return true; }
                if (!mbar_wait_warp(bar(L::B_Q), s_items & 1, abort_flag)) return false;
                ++s_items;
            }
            const int st = t % NS;
            if (!mbar_wait_warp(bar(L::B_KF + st), (t / NS) & 1, abort_flag)) return false;
#pragma unroll 1
            for (int X = 0; X < kGroups; ++X) {
                if constexpr (!L::kAlias) {               // the unit before has its scores in registers
                    const int before = t * kGroups + X - 1;
                    if (before >= 0 && !mbar_wait_warp(bar(L::B_SFREE + before % kGroups), (before / kGroups) & 1, abort_flag))
                        return false;
                }
                tc_fence_after();
                const uint64_t a = dQ + (uint64_t)((X * L::kTile) >> 4);
                const uint64_t b = dK + (uint64_t)((st * L::kTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
                    mma_ss_elect(tmem, a + o, b + o, kIdescQK, kk > 0 ? 1u : 0u);
                }
                commit_elect(bar(L::B_S + X));
            }
            commit_elect(bar(L::B_KE + st));
            return true;
        };
        auto issue_pv = [&](int t) -> bool {
            if (t == v_end) {
                if (!mbar_wait_warp(bar(L::B_ITEM + v_items % kItemNotes), (v_items / kItemNotes) & 1, abort_flag)) return false;
                v_first = t;
                v_end = t + notes[v_items % kItemNotes].run;
                if (v_end == t) { v_done = true; return true; }
                ++v_items;
            }
            const int st = t % NS;
            if (!mbar_wait_warp(bar(L::B_VF + st), (t / NS) & 1, abort_flag)) return false;
#pragma unroll 1
            for (int X = 0; X < kGroups; ++X) {
                if (!mbar_wait_warp(bar(L::B_P + X), t & 1, abort_flag)) return false;
                tc_fence_after();
                const uint64_t b = dV + (uint64_t)((st * L::kTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ts_elect(tmem + L::TM_O + (uint32_t)D * X, tmem + L::TM_P + 64u * X + kk * 8,
                                 b + (uint64_t)(kk * (2048 >> 4)), kIdescPV, kk > 0 || t > v_first ? 1u : 0u);
                if constexpr (!L::kAlias) commit_elect(bar(L::B_PV + X));
                if (t + 1 == v_end) commit_elect(bar(L::B_ODONE + X));
            }
            commit_elect(bar(L::B_VE + st));
            return true;
        };
        bool ok = true;
        int t = 0;
        if constexpr (kGroups == 2) {
            if (warp == L::kWarpIssue) {
                for (; ok && !s_done; ++t) ok = issue_s(t);
            } else {
                for (; ok && !v_done; ++t) ok = issue_pv(t);
            }
        } else if constexpr (L::kAlias) {
            for (; ok && !v_done; ++t) ok = issue_s(t) && issue_pv(t);
        } else {
            // the scores of the next tile before this one's product
            ok = issue_s(0);
            for (; ok && !v_done; ++t) ok = (s_done || issue_s(t + 1)) && issue_pv(t);
        }
        if (!ok && lane == 0) fail(R_ISSUE, t);
        const int drain = L::B_DRAIN + warp - L::kWarpIssue;
        commit_elect(bar(drain));                         // all products done before teardown
        const int zero = 0;
        mbar_wait_warp(bar(drain), 0, &zero);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == L::kWarpIssue) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
}

// ---------------------------------------------------------------------------
// Join the items that a worker boundary cuts (list without shared prefix
// items; whole items were written by the kernel above).  blockIdx.x + 1 is
// the worker behind the boundary, blockIdx.y a group of 16 rows.  Bound by
// latency, so kFlight parts of a row are loaded together.
// ---------------------------------------------------------------------------
template <int D, int M>
__global__ void __launch_bounds__(256) paged_cuts_kernel(const __grid_constant__ PagedParams p) {
    constexpr int V = D / 32, kRows = 2, kFlight = 4;      // channels of a lane, rows of a warp, parts in flight
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.x + 1;
    pdl_trigger();
    pdl_wait();
    const PagedCut cut = p.cuts[w];
    if (cut.b < 0) return;
    const PagedSched<M, 128, false> s(p);
    const int r0 = ((int)blockIdx.y * 8 + warp) * kRows;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        int b, i, hq;
        if (!paged_row(s, cut.b, cut.h, cut.rt, cut.n, r0 + k, b, i, hq)) continue;
        float acc[V], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 1
        for (int j0 = 0; j0 < cut.parts; j0 += kFlight) {
            float2 ml[kFlight];
            float y[kFlight][V];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {            // part 0: the second slot of worker w - 1
                const int j = j0 + f;
                const int64_t q = (int64_t)(j == 0 ? 2 * (w - 1) + 1 : 2 * (w - 1 + j)) * M + r0 + k;
                ml[f] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int v = 0; v < V; ++v) y[f][v] = 0.f;
                if (j < cut.parts) {
                    ml[f] = p.part_ml[q];
                    const float* src = p.part_o + q * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 x = *reinterpret_cast<const float4*>(src);
                        y[f][0] = x.x; y[f][1] = x.y; y[f][2] = x.z; y[f][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2*>(src);
                        y[f][0] = x.x; y[f][1] = x.y;
                    }
                }
            }
            float mn = m;
#pragma unroll
            for (int f = 0; f < kFlight; ++f) mn = fmaxf(mn, ml[f].x);
            const float ms = mn == -INFINITY ? 0.f : mn;
            const float fa = ex2_approx(m - ms);
            l *= fa;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= fa;
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const float fb = ex2_approx(ml[f].x - ms);
                l += ml[f].y * fb;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] += y[f][v] * fb;
            }
            m = mn;
        }
        const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
        uint16_t* dst = p.o + b * p.osb + hq * p.osh + i * p.osn + lane * V;
        const uint32_t lo = pack2(acc[0] * inv, acc[1] * inv);
        if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, pack2(acc[V - 2] * inv, acc[V - 1] * inv));
        else *reinterpret_cast<uint32_t*>(dst) = lo;
    }
}

template <int D, int kGroups, int kForm>
cudaError_t launch_one(const PagedParams& p, const CUtensorMap& tq, const CUtensorMap& tqp, const CUtensorMap& tk,
                       const CUtensorMap& tv, cudaStream_t s) {
    using L = TilesShape<D, kGroups>;
    static bool ready[64] = {};
    cudaError_t e = launch_pdl(paged_tiles_kernel<D, kGroups, kForm>, dim3((unsigned)p.workers), dim3(L::kThreads), L::kSmem, s, 1, true, ready,
                               tq, tqp, tk, tv, p);
    if (e != cudaSuccess) return e;
    if (kForm == F_LIST && p.workers > 1) {
        static bool cuts_ready[64] = {};
        e = launch_pdl(paged_cuts_kernel<D, L::M>, dim3((unsigned)p.workers - 1, L::M / 16), dim3(256), 0, s, 1, true, cuts_ready, p);
    }
    return e;
}

template <int D, int kGroups>
cudaError_t launch_form(int form, const PagedParams& p, const CUtensorMap& tq, const CUtensorMap& tqp, const CUtensorMap& tk,
                        const CUtensorMap& tv, cudaStream_t s) {
    if (form == F_ITEM) return launch_one<D, kGroups, F_ITEM>(p, tq, tqp, tk, tv, s);
    if (form == F_PREFIX) return launch_one<D, kGroups, F_PREFIX>(p, tq, tqp, tk, tv, s);
    return launch_one<D, kGroups, F_LIST>(p, tq, tqp, tk, tv, s);
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedParams& p, int D, int groups, const CUtensorMap& tq, const CUtensorMap& tqp,
                               const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    const int form = p.whole ? F_ITEM : p.pre_rt > 0 ? F_PREFIX : F_LIST;
    if (D == 64)
        return groups == 1 ? launch_form<64, 1>(form, p, tq, tqp, tk, tv, s) : launch_form<64, 2>(form, p, tq, tqp, tk, tv, s);
    return groups == 1 ? launch_form<128, 1>(form, p, tq, tqp, tk, tv, s) : launch_form<128, 2>(form, p, tq, tqp, tk, tv, s);
}

}  // namespace sage
