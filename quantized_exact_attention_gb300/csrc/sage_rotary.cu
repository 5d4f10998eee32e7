// sage_rotary.cu - rotary positions: rotation of queries (or of gradients), and
// the append to a page cache that rotates keys on their way into it.
//
// Pair j of a head's first R channels is turned by the angle a = pos * f_j:
//     y1 = A (x1 cos a - x2 sin a),   y2 = A (x1 sin a + x2 cos a)
// (inverse: -a, which is the transposed matrix and so the gradient).  The angle
// is held in turns of 2^-64: pos * round(f_j / (2 pi) * 2^64) modulo 2^64 is an
// integer product that wraps by itself: the error is below |pos| * 2^-64 turns
// from the frequency and 2^-32 from taking the upper half, so below 2^-31 turns
// at every position of 32 bits, where an FP32 product pos * f_j would be off by
// 0.06 rad at pos = 10^6.  Sine and cosine are FP32 of that angle, the products and their
// sum FP32; the result is rounded to BF16 once.
#include <algorithm>
#include <cmath>

#include "sage_gb300.h"
#include "sage_internal.h"
#include "sage_paged.h"
#include "sage_paged_sched.cuh"

namespace sage {
namespace {

// A lane holds the same two 16-byte chunks of the heads it takes, so it
// computes the sines and cosines of its 8 pairs once for all of them:
//   half layout         pair j = channels j and R/2 + j: chunks u and u + R/16
//                       are the first and the second channels of pairs 8u..8u+7
//   interleaved layout  pair j = channels 2j and 2j + 1: a chunk holds 4 pairs;
//                       the same two chunks hold pairs 4u.. and 4(u + R/16)..
//   channels >= R       units behind R/16 copy two chunks each
// D/16 lanes hold a head, up to 2^slot_shift heads of a token lie beside each
// other, and what is left of a warp's 32 lanes takes further tokens.  A lane has
// the chunks of kFlight heads in flight: of one token, or where a token has too
// few, of kTokens tokens (one head of 393,216 tokens, 201 MB: 62.6 us with a
// token at a time, 51.7 so, and 44.6 with the sines below in place of
// sincospif: 64 of them for every 512 bytes).
struct Turn {
    const int32_t* positions;            // [B][pos_stride] or null: the token's number
    const int32_t* start;                // [B] or null: 0
    const uint64_t* turns;               // [R/2]
    int64_t pos_stride;
    float amplitude;
    int inverse;
    int rot_units;                       // R / 16
    int unit_shift, slot_shift;          // log2 of D/16 and of the heads beside each other
    int splits, heads_each;              // warps that share a token's heads, heads of one
    int64_t tokens;                      // B * N, below 2^31
    int N, H;
    FastDiv by_N;
};

// What a lane has to do.
struct LaneWork {
    int64_t first;                       // its first token; the next one is `apart` behind
    int apart;
    int unit, c0, c1;                    // its unit and the channels its two chunks begin at
    int h0, h1, step;                    // heads h0, h0 + step, ... below h1
    bool rotates;
};

constexpr int kRotaryThreads = 256;

template <int kTokens>
__device__ __forceinline__ LaneWork lane_work(const Turn& p) {
    LaneWork x;
    const int64_t warp = (int64_t)blockIdx.x * (kRotaryThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, slots = 1 << p.slot_shift, units = 1 << p.unit_shift;
    const uint32_t group = p.splits == 1 ? (uint32_t)warp : (uint32_t)warp / (uint32_t)p.splits;
    const int split = (int)((uint32_t)warp - group * (uint32_t)p.splits);
    x.apart = 32 >> (p.unit_shift + p.slot_shift);
    x.first = (int64_t)group * kTokens * x.apart + (lane >> (p.unit_shift + p.slot_shift));
    x.unit = lane & (units - 1);
    x.rotates = x.unit < p.rot_units;
    const int between = x.rotates ? p.rot_units : units - p.rot_units;
    const int chunk = x.rotates ? x.unit : p.rot_units + x.unit;         // chunks 2 rot_units.. are copied
    x.c0 = chunk * 8;
    x.c1 = (chunk + between) * 8;
    x.h0 = split * p.heads_each + ((lane >> p.unit_shift) & (slots - 1));
    x.h1 = min(p.H, (split + 1) * p.heads_each);
    x.step = slots;
    return x;
}

// Position of token i of request b.
__device__ __forceinline__ int64_t position(const Turn& p, int b, int i) {
    return (p.start == nullptr ? 0 : (int64_t)p.start[b]) +
           (p.positions == nullptr ? (int64_t)i : (int64_t)p.positions[b * p.pos_stride + i]);
}

// Sine and cosine of an angle of phase * 2^-32 turns.  The angle is folded to x
// in [-pi/4, pi/4] about the nearest quarter turn; there the Taylor series up to
// x^9 and x^8 leave x^11 / 11! < 2e-9 and x^10 / 10! < 3e-8.  x is off by three
// roundings (3 * 2^-24 of it, times a slope of cos x: 1.0e-7 at most), the sums
// by one and what is left of those inside (4e-8): both within 2^-22 in all.
__device__ __forceinline__ void sincos_turns(uint32_t phase, float& sn, float& cs) {
    const uint32_t y = phase + 0x20000000u;                // upper two bits: the nearest quarter turn
    const float x = (float)(int)((y & 0x3fffffffu) - 0x20000000u) * (float)(6.283185307179586 * 0x1p-32);
    const float z = x * x;
    float u = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    u = fmaf(z, u, 1.f / 120.f);
    u = fmaf(z, u, -1.f / 6.f);
    const float si = fmaf(x * z, u, x);
    float v = fmaf(z, 1.f / 40320.f, -1.f / 720.f);
    v = fmaf(z, v, 1.f / 24.f);
    v = fmaf(z, v, -0.5f);
    const float co = fmaf(z, v, 1.f);
    const bool odd = y & 0x40000000u;
    sn = __uint_as_float(__float_as_uint(odd ? co : si) ^ (y & 0x80000000u));
    cs = __uint_as_float(__float_as_uint(odd ? si : co) ^ ((y + 0x40000000u) & 0x80000000u));
}

// Cosines and sines (times the amplitude) of the lane's pairs at a position.
template <bool kInterleaved>
__device__ __forceinline__ void lane_angles(const Turn& p, const LaneWork& x, int64_t pos, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const int j = kInterleaved ? 4 * (e < 4 ? x.unit : x.unit + p.rot_units) + (e & 3) : 8 * x.unit + e;
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(p.turns + j);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t phase = (uint32_t)(((uint64_t)pos * (k == 0 ? f.x : f.y)) >> 32);
            if (p.inverse) phase = 0u - phase;
            float sn, cs;
            sincos_turns(phase, sn, cs);
            c[e + k] = cs * p.amplitude;
            s[e + k] = sn * p.amplitude;
        }
    }
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool kInterleaved>
__device__ __forceinline__ void rotate(uint4& va, uint4& vb, const float (&c)[8], const float (&s)[8]) {
    uint32_t a[4] = {va.x, va.y, va.z, va.w}, b[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a0 = lo_bf16(a[k]), a1 = hi_bf16(a[k]), b0 = lo_bf16(b[k]), b1 = hi_bf16(b[k]);
        if (kInterleaved) {
            a[k] = two_bf16(a0 * c[k] - a1 * s[k], a0 * s[k] + a1 * c[k]);
            b[k] = two_bf16(b0 * c[4 + k] - b1 * s[4 + k], b0 * s[4 + k] + b1 * c[4 + k]);
        } else {
            a[k] = two_bf16(a0 * c[2 * k] - b0 * s[2 * k], a1 * c[2 * k + 1] - b1 * s[2 * k + 1]);
            b[k] = two_bf16(a0 * s[2 * k] + b0 * c[2 * k], a1 * s[2 * k + 1] + b1 * c[2 * k + 1]);
        }
    }
    va = make_uint4(a[0], a[1], a[2], a[3]);
    vb = make_uint4(b[0], b[1], b[2], b[3]);
}

// ---------------------------------------------------------------------------
// Rotation of a [B, H, N, D] view: each row read and written once, HBM bounds
// it.  The first rows are on their way while the angles are computed (24 heads
// of 16,384 tokens, 201 MB: 31.1 us, 0.95 of the copy rate; the angles first
// 33.4).  Three blocks an SM hold eight chunks a lane in flight in registers
// (four blocks with four chunks 31.5; eight chunks that spill 39.0).
// ---------------------------------------------------------------------------
struct RopeParams {
    Turn turn;
    const uint16_t* x;
    uint16_t* o;
    int64_t xsb, xsh, xsn, osb, osh, osn;
    const int32_t* n_len;                // or null: N
    int in_place;
};

template <bool kInterleaved, int kTokens>
__global__ void __launch_bounds__(kRotaryThreads, 3) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kFlight = 4, kHeads = kFlight / kTokens; // heads whose loads precede their stores, of a token
    pdl_trigger();
    pdl_wait();
    const LaneWork w = lane_work<kTokens>(p.turn);
    if (p.in_place && !w.rotates) return;
    const uint16_t* x[kTokens];
    uint16_t* o[kTokens];
    int b0 = 0, i0 = 0;                                    // request and token (of one alone)
    int64_t pos[kTokens];
    bool live[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
        const int64_t n = w.first + t * w.apart;
        const int b = fast_div((int)min(n, p.turn.tokens - 1), p.turn.by_N), i = (int)(n - (int64_t)b * p.turn.N);
        live[t] = n < p.turn.tokens && (p.n_len == nullptr || i < p.n_len[b]);
        x[t] = p.x + b * p.xsb + i * p.xsn;
        o[t] = p.o + b * p.osb + i * p.osn;
        if (kTokens > 1) pos[t] = live[t] && w.rotates ? position(p.turn, b, i) : 0;
        b0 = b; i0 = i;
    }
    if (kTokens == 1 && !live[0]) return;
    uint4 a[kFlight], b[kFlight];
    auto load = [&](int h0) {
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int t = k / kHeads, h = h0 + (k % kHeads) * w.step;
            if (live[t] && h < w.h1) {
                a[k] = *reinterpret_cast<const uint4*>(x[t] + h * p.xsh + w.c0);
                b[k] = *reinterpret_cast<const uint4*>(x[t] + h * p.xsh + w.c1);
            }
        }
    };
    load(w.h0);
    float c[8], s[8];
    // a token alone: its position is asked for behind its rows (before them: 32.7 us in place of 31.1)
    if (kTokens == 1 && w.rotates) lane_angles<kInterleaved>(p.turn, w, position(p.turn, b0, i0), c, s);
#pragma unroll 1
    for (int h0 = w.h0;;) {
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int t = k / kHeads, h = h0 + (k % kHeads) * w.step;
            if (kTokens > 1 && k % kHeads == 0 && live[t] && w.rotates) lane_angles<kInterleaved>(p.turn, w, pos[t], c, s);
            if (live[t] && h < w.h1) {
                if (w.rotates) rotate<kInterleaved>(a[k], b[k], c, s);
                *reinterpret_cast<uint4*>(o[t] + h * p.osh + w.c0) = a[k];
                *reinterpret_cast<uint4*>(o[t] + h * p.osh + w.c1) = b[k];
            }
        }
        if (kTokens > 1) break;                            // they have no more heads
        h0 += kFlight * w.step;
        if (h0 >= w.h1) break;
        load(h0);
    }
}

// ---------------------------------------------------------------------------
// Append with rotation: K rotated, V copied, into the cache rows of the slots.
// HBM bounds it (16 ragged prompts of up to 2,048 tokens, 16 heads of 128
// channels, 259 MB: 40.6 us, 0.94 of the copy rate; the angles before the first
// loads 42.9; four blocks an SM with half the chunks in flight 41.4).
// ---------------------------------------------------------------------------
struct AppendRopeParams {
    Turn turn;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* ck;
    uint16_t* cv;
    const int32_t* slots;
    int* status;
    int64_t ksb, ksh, ksn, vsb, vsh, vsn;
    int64_t ckp, ckh, ckt, cvp, cvh, cvt;
    int64_t slots_stride, capacity;
    int page, page_shift;
};

template <bool kInterleaved, int kTokens>
__global__ void __launch_bounds__(kRotaryThreads, 3) append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int kFlight = 2, kHeads = kFlight / kTokens; // heads whose loads precede their stores, of a token
    pdl_trigger();
    pdl_wait();
    const LaneWork w = lane_work<kTokens>(p.turn);
    int b0 = 0, i0 = 0, slot[kTokens];                     // request and token (of one alone), places in the cache
    int64_t pos[kTokens];
    const uint16_t* kr[kTokens];
    const uint16_t* vr[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
        const int64_t n = w.first + t * w.apart;
        const int b = fast_div((int)min(n, p.turn.tokens - 1), p.turn.by_N), i = (int)(n - (int64_t)b * p.turn.N);
        slot[t] = n < p.turn.tokens ? p.slots[b * p.slots_stride + i] : -1;
        if (kTokens > 1) pos[t] = n < p.turn.tokens && w.rotates ? position(p.turn, b, i) : 0;
        b0 = b; i0 = i;
        kr[t] = p.k + b * p.ksb + i * p.ksn;
        vr[t] = p.v + b * p.vsb + i * p.vsn;
    }
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
        if (slot[t] >= p.capacity) {
            if (w.unit == 0 && atomicCAS(p.status, 0, kErrPage) == 0) p.status[3] = slot[t] >> p.page_shift;
            slot[t] = -1;
        }
    if (kTokens == 1 && slot[0] < 0) return;
    uint4 a[kFlight], b[kFlight], d[kFlight], e[kFlight];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int t = u / kHeads, h = h0 + (u % kHeads) * w.step;
            if (slot[t] >= 0 && h < w.h1) {
                a[u] = *reinterpret_cast<const uint4*>(kr[t] + h * p.ksh + w.c0);
                b[u] = *reinterpret_cast<const uint4*>(kr[t] + h * p.ksh + w.c1);
                d[u] = *reinterpret_cast<const uint4*>(vr[t] + h * p.vsh + w.c0);
                e[u] = *reinterpret_cast<const uint4*>(vr[t] + h * p.vsh + w.c1);
            }
        }
    };
    load(w.h0);
    float c[8], s[8];
    if (kTokens == 1 && w.rotates) lane_angles<kInterleaved>(p.turn, w, position(p.turn, b0, i0), c, s);
#pragma unroll 1
    for (int h0 = w.h0;;) {
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int t = u / kHeads, h = h0 + (u % kHeads) * w.step;
            if (kTokens > 1 && slot[t] >= 0 && w.rotates) lane_angles<kInterleaved>(p.turn, w, pos[t], c, s);
            if (slot[t] >= 0 && h < w.h1) {
                const int64_t pg = slot[t] >> p.page_shift;
                const int off = slot[t] & (p.page - 1);
                uint16_t* ck = p.ck + pg * p.ckp + off * p.ckt + h * p.ckh;
                uint16_t* cv = p.cv + pg * p.cvp + off * p.cvt + h * p.cvh;
                *reinterpret_cast<uint4*>(cv + w.c0) = d[u];
                *reinterpret_cast<uint4*>(cv + w.c1) = e[u];
                if (w.rotates) rotate<kInterleaved>(a[u], b[u], c, s);
                *reinterpret_cast<uint4*>(ck + w.c0) = a[u];
                *reinterpret_cast<uint4*>(ck + w.c1) = b[u];
            }
        }
        if (kTokens > 1) break;                            // they have no more heads
        h0 += kFlight * w.step;
        if (h0 >= w.h1) break;
        load(h0);
    }
}

// Fill `t`; the grid's warps in *warps and how many tokens a lane has in flight
// (of `flight` heads) in *together.  SAGE_OK or why the call is refused.
int make_turn(Turn& t, int64_t& warps, int& together, int flight, const sage_rotary* r, const int32_t* positions,
              int64_t positions_stride, const int32_t* start, int B, int H, int N, int D, int inverse) {
    if (r == nullptr || r->turns == nullptr || r->rotary_dim <= 0 || positions_stride < 0) return SAGE_ERR_ARG;
    if (r->rotary_dim > D || r->rotary_dim % 16 || !aligned16(r->turns)) return SAGE_ERR_UNSUPPORTED;
    if ((int64_t)B * N > INT32_MAX) return SAGE_ERR_UNSUPPORTED;
    t.positions = positions; t.pos_stride = positions_stride; t.start = start;
    t.turns = r->turns; t.amplitude = r->amplitude; t.inverse = inverse != 0;
    t.rot_units = r->rotary_dim / 16;
    t.tokens = (int64_t)B * N; t.N = N; t.H = H;
    t.by_N = make_fast_div((uint32_t)N);
    t.unit_shift = D == 128 ? 3 : 2;
    t.slot_shift = 0;
    while (t.slot_shift < 5 - t.unit_shift && (1 << t.slot_shift) < H) ++t.slot_shift;
    const int apart = 32 >> (t.unit_shift + t.slot_shift);
    const int passes = (int)ceil_div(H, 1 << t.slot_shift);
    const int64_t fill = 24 * std::max(1, sm_count());     // warps that fill the GPU
    together = 1;
    while (2 * together * passes <= flight && ceil_div(t.tokens, apart * 2 * together) >= fill) together *= 2;
    const int64_t groups = ceil_div(t.tokens, apart * together);
    const int want = (int)std::min<int64_t>(passes, ceil_div(fill, groups));
    t.heads_each = (int)ceil_div(passes, want) << t.slot_shift;
    t.splits = (int)ceil_div(H, t.heads_each);
    warps = groups * t.splits;
    return SAGE_OK;
}

template <bool kInterleaved>
cudaError_t launch_rope(const RopeParams& p, int together, int64_t warps, cudaStream_t s) {
    static bool ready[3][64] = {};
    const dim3 grid((unsigned)ceil_div(warps, kRotaryThreads / 32)), block(kRotaryThreads);
    if (together == 4) return launch_pdl(rope_kernel<kInterleaved, 4>, grid, block, 0, s, 1, false, ready[2], p);
    if (together == 2) return launch_pdl(rope_kernel<kInterleaved, 2>, grid, block, 0, s, 1, false, ready[1], p);
    return launch_pdl(rope_kernel<kInterleaved, 1>, grid, block, 0, s, 1, false, ready[0], p);
}
template <bool kInterleaved>
cudaError_t launch_append(const AppendRopeParams& p, int together, int64_t warps, cudaStream_t s) {
    static bool ready[2][64] = {};
    const dim3 grid((unsigned)ceil_div(warps, kRotaryThreads / 32)), block(kRotaryThreads);
    if (together == 2) return launch_pdl(append_rope_kernel<kInterleaved, 2>, grid, block, 0, s, 1, false, ready[1], p);
    return launch_pdl(append_rope_kernel<kInterleaved, 1>, grid, block, 0, s, 1, false, ready[0], p);
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_rotary_turns(const double* frequencies, int n, uint64_t* turns) {
    if (frequencies == nullptr || turns == nullptr || n <= 0) return SAGE_ERR_ARG;
    // 1 / (2 pi) as the sum of two doubles, so that the 64 bits behind the whole turns are right
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    for (int j = 0; j < n; ++j) {
        const double f = std::fabs(frequencies[j]);
        if (!(f < 0x1p20)) return SAGE_ERR_ARG;                            // NaN too
        const double turn = f * kHi, rest = std::fma(f, kHi, -turn) + f * kLo;
        const double part = turn - std::floor(turn);                       // whole turns a position do not matter
        const double upper = std::ldexp(part, 32), whole = std::floor(upper);
        const uint64_t t = ((uint64_t)whole << 32) + (uint64_t)std::llrint(std::ldexp(upper - whole, 32) + std::ldexp(rest, 64));
        turns[j] = frequencies[j] < 0.0 ? 0 - t : t;
    }
    return SAGE_OK;
}

int sage_rope(const sage_tensor* x, const sage_tensor* out, int B, int H, int N, int D, const int32_t* positions,
              int64_t positions_stride, const int32_t* start, const int32_t* n_len, const sage_rotary* rotary, int inverse,
              void* stream) {
    int rc;
    if ((rc = check_view(x)) != SAGE_OK || (rc = check_view(out)) != SAGE_OK) return rc;
    if (B <= 0 || H <= 0 || N <= 0) return SAGE_ERR_ARG;
    if (D != 64 && D != 128) return SAGE_ERR_UNSUPPORTED;
    // rows written once: no broadcast axis
    if ((B > 1 && out->stride_b < D) || (H > 1 && out->stride_h < D) || (N > 1 && out->stride_n < D))
        return SAGE_ERR_UNSUPPORTED;
    const bool in_place = x->ptr == out->ptr;
    if (in_place && ((B > 1 && x->stride_b != out->stride_b) || (H > 1 && x->stride_h != out->stride_h) ||
                     (N > 1 && x->stride_n != out->stride_n)))
        return SAGE_ERR_ARG;
    RopeParams p{};
    int64_t warps = 0;
    int together = 1;
    if ((rc = make_turn(p.turn, warps, together, 4, rotary, positions, positions_stride, start, B, H, N, D, inverse)) != SAGE_OK)
        return rc;
    p.x = static_cast<const uint16_t*>(x->ptr);
    p.o = static_cast<uint16_t*>(const_cast<void*>(out->ptr));
    p.xsb = x->stride_b; p.xsh = x->stride_h; p.xsn = x->stride_n;
    p.osb = out->stride_b; p.osh = out->stride_h; p.osn = out->stride_n;
    p.n_len = n_len; p.in_place = in_place;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((rotary->interleaved ? launch_rope<true>(p, together, warps, s) : launch_rope<false>(p, together, warps, s)) != cudaSuccess)
        return SAGE_ERR_LAUNCH;
    set_last_launch_count(1);
    return SAGE_OK;
}

int sage_cache_append_rope(const sage_tensor* k, const sage_tensor* v, int B, int N, const int32_t* slots,
                           int64_t slots_stride, const int32_t* positions, int64_t positions_stride, const int32_t* start,
                           const sage_rotary* rotary, const sage_page_cache* cache, void* stream) {
    int rc = check_page_cache(cache);
    if (rc != SAGE_OK) return rc;
    if (B <= 0 || N <= 0 || slots == nullptr || slots_stride < 0) return SAGE_ERR_ARG;
    if ((rc = check_view(k)) != SAGE_OK || (rc = check_view(v)) != SAGE_OK) return rc;
    AppendRopeParams p{};
    int64_t warps = 0;
    int together = 1;
    if ((rc = make_turn(p.turn, warps, together, 2, rotary, positions, positions_stride, start, B, cache->heads, N, cache->D, 0)) !=
        SAGE_OK)
        return rc;
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
    p.page = cache->page_size;
    p.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((rotary->interleaved ? launch_append<true>(p, together, warps, s) : launch_append<false>(p, together, warps, s)) !=
        cudaSuccess)
        return SAGE_ERR_LAUNCH;
    set_last_launch_count(1);
    return SAGE_OK;
}

}  // extern "C"
