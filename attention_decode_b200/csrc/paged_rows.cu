// Attention over the paged 8-bit cache for many query rows: prompts, and
// chunks of prompts behind a context (bf16 queries and outputs).
//
// A unit is 256 (query row, head) pairs of one sequence and kv-head, heads
// fastest, in two halves of 128 rows; a row is a TMEM lane and one thread's.
// Per tile of 128 tokens and half:
//   S = Q K^T      tcgen05.mma kind::f8f6f4: K as the cache holds it, Q as two
//                  pieces in one accumulator: an e4m3 one of 4 significant bits,
//                  and what it leaves in e5m2 (of the 8 bits of a bf16 query the
//                  4 below have 3 significant ones, and e5m2 reaches down to
//                  2^-16). With a row scaled to at most 448, that is an element
//                  down to 2^-6 exactly, and a smaller one up to 2^-14,
//   p = 2^(s - m)  one thread per row: no value crosses a thread,
//   O += P V       kind::f16, P from TMEM (over S), V widened to fp16 (exact)
//                  in shared memory by a warpgroup of its own.
// fp16 weights keep 11 bits; the running maximum may lag by 2^kLag and the
// bias 2^kBias keeps the largest below 2^15.75 and steps at 2^-23 of the largest.
// What meets V's codes is a weight times its page's v scale, over a reference
// of the row's own: the largest such product among the tokens that the row has
// seen has a reference of its own lag and takes the range of fp16 as above,
// whatever the scales are; the sum of the weights stays on their own maximum. No
// bit of a row depends on what it does not see: a warp's rows raise their maxima
// together while all of them have seen the same tokens (every tile so far was
// whole), from then on each by itself. (A raise holds up its half's P V; rows that
// raise one by one do so at more steps: the 8192 prompt below took 724 us.)
//
// What bounds it: a tile needs 2048 clocks of the tensor cores (2 halves x (S
// 512 + P V 512)) and 2048 of the exponential unit (2 x 16384 at 16 a clock), and
// takes ~4900: each is busy 40 % of the time, the issue slots 50 %. A row warp's
// own chain (scores from TMEM, exponents, weights back, 64 tokens at a time) is
// 1840 clocks long where the exponential unit alone would allow 512, and an SM
// sub-partition has two such warps. Measured: a prompt of 8192 tokens, 32 query
// heads on 8 kv-heads, causal, 693 to 708 us (778 TFLOP/s, 47 % of the measured bf16
// rate); 447 + 280 rows behind 21.5k and 16.8k tokens 292 to 308 us (774 TFLOP/s);
// 4 prompts of ~1500 under a 511 window with 5 sinks 157 to 163 us. On the way: scores
// in one go per tile 929 us, then 64-token steps with the next scores in flight
// and MMA issue under elect (before, the issuing thread alone took 1700 clocks
// per half and step) 749 us. Tried: two threads per row (794 us with, 822
// without a register split; the second barrier per step and spills cost what
// the overlap gains), the scores of the next chunk loaded ahead (735-760 us).
#include <math.h>

#include "f32x2.cuh"
#include "paged_join.cuh"

namespace nsnq {

namespace {

constexpr int RC = 256;         // rows of a unit
constexpr int kThreads = 512;   // warps 0-3, 4-7: rows; 8-11: V to fp16; 12: TMA; 13: MMA issue
constexpr float kLag = 16.75f, kBias = -1.f;
constexpr int kKStages = 3, kRing = 8;
constexpr int kMaxSlots = 8;
// Tiles that a unit's queries and epilogue cost (2, 3, 5, 8: the 8192 prompt 795,
// 733, 689, 695 us; short windows 143, 144, 147, 148 us).
constexpr int kSetup = 5;

// shared memory, from a 1024-aligned base
constexpr uint32_t kQ = 0;                        // [half][piece][128 rows][128 B]
constexpr uint32_t kK = kQ + 4 * 16384;           // [stage][128 tokens][128 B]
constexpr uint32_t kV = kK + kKStages * 16384;    // [2][128 tokens][128 B]
constexpr uint32_t kV16 = kV + 2 * 16384;         // [2][channel half][128 tokens][128 B]
constexpr uint32_t kMisc = kV16 + 4 * 16384;

struct Misc {
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[2], v_empty[2], w_full[2], w_free[2], sc_full[kRing];
    uint64_t q_ready[2], s_full[2][2], p_full[2][2], pv_done[2], o_full[2], done;
    uint32_t tmem;
    PagedRange range;
    uint32_t ok[kRing];                // pages of the tile that were loaded
    float2 scale[kRing][kMaxSlots];    // (k scale, v scale) of a page
    uint32_t nan[RC][4];               // row: channels that a NaN code of a partly seen tile reaches
};

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two e5m2 codes (nearest, ties to even, held at the largest value); the low byte holds a.
__device__ __forceinline__ uint32_t e5m2x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Queries of the warp's 32 rows (from unit row `first` on) as two pieces,
// eight lanes to a row, 16 channels each; returns the scale of this lane's row.
__device__ __forceinline__ float write_rows(const PagedAttnArgs& a, const PagedUnit& u, int h, int first, uint8_t* hi,
                                            int lrow0) {
    const int lane = lane_id(), c = lane & 7, G = (int)a.G.d;
    float mine = 0.f;
    uint4 raw[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // every load first: their latencies overlap
        const int r = first + 4 * i + (lane >> 3);
        raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
        if (r < u.rows) {
            const int rr = u.r0 + r, qi = (int)fdiv((uint32_t)rr, a.G);
            const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                            (int64_t)(u.row0 + qi) * a.q_st +
                                                            (int64_t)(h * G + rr - qi * G) * a.q_sh + 16 * c);
            raw[i][0] = q[0];
            raw[i][1] = q[1];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 w0 = raw[i][0], w1 = raw[i][1];
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        float x[16];
        float top = 0.f;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            top = fmaxf(top, fabsf(x[k]));
            bad |= !isfinite(x[k]);
        }
#pragma unroll
        for (int m = 4; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, m));
        bad = ((__ballot_sync(kFull, bad) >> (lane & 24)) & 0xffu) != 0;
        // the least e >= -126 with top <= 448 * 2^e
        const uint32_t bits = __float_as_uint(top);
        int e = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) > 0x600000u ? 7 : 8);
        e = bad ? 0 : (e < -126 ? -126 : e);
        const float scale = __shfl_sync(kFull, __uint_as_float((uint32_t)(127 + e) << 23), (lane & 3) << 3);
        if ((lane >> 2) == i) mine = scale;
        float up = __uint_as_float((uint32_t)(127 - e) << 23);
        if (a.scale_log2 < 0.f) up = -up;
        uint32_t p[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) y[m] = x[4 * k + m] * up;
            const uint32_t c0 = e4m3x2(y[0], y[1]), c1 = e4m3x2(y[2], y[3]);
            const uint32_t h0 = e4m3x2_to_f16x2(c0), h1 = e4m3x2_to_f16x2(c1);
            p[k] = bad ? 0x7f7f7f7fu : (c0 | (c1 << 16));
            l[k] = bad ? 0u : (e5m2x2(y[0] - f16_lo(h0), y[1] - f16_hi(h0)) |
                               (e5m2x2(y[2] - f16_lo(h1), y[3] - f16_hi(h1)) << 16));
        }
        const int lrow = lrow0 + 4 * i + (lane >> 3), at = lrow * 128 + ((c ^ (lrow & 7)) << 4);
        *reinterpret_cast<uint4*>(hi + at) = make_uint4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<uint4*>(hi + 16384 + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
    return mine * fabsf(a.scale_log2);
}

// A row's view of a tile: columns up to hi and above lo, or below sink, on
// pages that were loaded.
struct View {
    int hi, lo, sink;
    uint32_t ok;
    int page_log;
    __device__ __forceinline__ static uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u; }
    __device__ __forceinline__ uint32_t bits(int c0) const {  // of columns c0 .. c0 + 31
        uint32_t b = below(hi + 1 - c0) & (~below(lo + 1 - c0) | below(sink - c0));
        if (!((ok >> (c0 >> page_log)) & 1u)) b &= 0xffff0000u;
        if (!((ok >> ((c0 + 16) >> page_log)) & 1u)) b &= 0xffffu;
        return b;
    }
};

// A row's running state in a segment.
struct RowState {
    float c;           // score scale (softmax scale, log2 e, query scale)
    float m, l;        // running maximum (log2 units), sum of 2^(s - m + kBias)
    float vref;        // reference of weight x v scale, relative to m; 0 before the first token
};

// The factor of weights under a page's v scale. (A finite one: a weight of 0
// stays 0. One that this holds down has passed kLag and raises the reference. The
// scale of a page that was not loaded is void, but then no weight is seen.)
__device__ __forceinline__ float reciprocal(float v) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(v));
    return inv;
}
__device__ __forceinline__ float value_factor(float vs, bool seen, float vref, float inv) {
    return !seen ? 0.f : vs == vref ? 1.f : fminf(vs * inv, 0x1p126f);
}

// The exponent that a weight may have under factor w: kBias + kLag, less the next
// whole log2 of a w above 1. (Known before the exponentials: their sum, times w,
// would do as well and comes later.)
__device__ __forceinline__ float weight_limit(float w) {
    const int n = max((int)((__float_as_uint(w) + 0x7fffffu) >> 23), 127);
    return kBias + kLag + 127.f - (__uint_as_float(0x4b000000u + n) - 0x1p23f);
}

// Multiplies a row's weights of the step so far (`done` columns of fp16 pairs) and,
// if there is one, its output by a factor.
__device__ __noinline__ void rescale_row(uint32_t s, int done, uint32_t o, bool have_o, float f) {
    tmem_wait_st();  // the weights so far may still be on their way
#pragma unroll 1
    for (int i = 0; i < done; i += 8) {
        uint32_t u[8];
        TmemLoad<8>::run(s + i, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = f16x2(f16_lo(u[k]) * f, f16_hi(u[k]) * f);
        tmem_st8(s + i, reinterpret_cast<float*>(u));
    }
#pragma unroll 1
    for (int i = 0; have_o && i < kD; i += 32) {
        uint32_t u[32];
        TmemLoad<32>::run(o + i, u);
#pragma unroll
        for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * f);
        tmem_st32(o + i, u);
    }
    tmem_wait_st();
}

// Weights of 16 columns of a row from their scores u: exponents, the largest
// of them, 2^x, their sum; packed in fp16 pairs, times w. WEIGH: some row's
// reference is not the page's v scale (w may not be 1). (Exponents are formed in
// packed pairs, as the scores lie; what follows 2^x is scalar: packing it again
// costs more moves than it saves.)
template <bool MASKED, bool WEIGH>
__device__ __forceinline__ void row_weights(const uint32_t (&u)[16], uint32_t seen, float ks, float w, const RowState& st,
                                            float& most, float& sum, uint32_t (&p)[8]) {
    const uint64_t nm = pk2(kBias - st.m, kBias - st.m);
    const float f = ks * st.c;
    const uint64_t f2 = pk2(f, f);
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        float2 x = upk2(fma2(pk2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), f2, nm));
        if (MASKED) {
            x.x = (seen >> i) & 1u ? x.x : -INFINITY;
            x.y = (seen >> i) & 2u ? x.y : -INFINITY;
        }
        top[(i >> 1) & 3] = fmaxf(top[(i >> 1) & 3], fmaxf(x.x, x.y));
        x.x = exp2_approx(x.x);
        x.y = exp2_approx(x.y);
        acc[(i >> 1) & 1] += x.x;
        acc[2 + ((i >> 1) & 1)] += x.y;
        if (WEIGH) {
            x.x *= w;
            x.y *= w;
        }
        p[i / 2] = f16x2(x.x, x.y);
    }
    most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Raises the maximum of the rows that need it to that of columns 16 q .. 63 of
// step b (their scores are still in TMEM), and the reference to the largest
// weight x v scale there, and scales those rows' weights and outputs so far;
// returns the new maximum and reference and the factor of the sum of weights. The
// reference is a page's v scale itself where the largest weight lies there
// (weights need no factor then), and from 2^-126 to 2^126: its reciprocal is a
// normal number.
// Calls are rare, but all warps of a half wait for one: of the step's columns
// rather than the 16 at hand, and with a wide lag, a third as many are needed.
__device__ __noinline__ float3 raise_row(uint32_t s, uint32_t o, bool have_o, int q, int b, uint32_t seen0, uint32_t seen1,
                                         const float2* scale, int page_log, float c, bool need, float m, float vref) {
    float mn = m, vn = 0.f;
#pragma unroll 1
    for (int i = q; i < 4; ++i) {
        const uint32_t seen = (i < 2 ? seen0 : seen1) >> (16 * (i & 1));
        const float2 kv = scale[(64 * b + 16 * i) >> page_log];
        const float f0 = kv.x * c;
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            tmem_ld<8>(s + 16 * i + 8 * h, v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if ((seen >> (8 * h + k)) & 1u) top = fmaxf(top, v[k] * f0);
        }
        if (need && top > -INFINITY) {  // vn is relative to mn
            const float up = fmaxf(mn, top);
            vn = fmaxf(mn == up ? vn : exp2_approx(mn - up) * vn, top == up ? kv.y : exp2_approx(top - up) * kv.y);
            mn = up;
        }
    }
    const float f = m == mn ? 1.f : exp2_approx(m - mn), old = vref * f;
    vn = need && mn > -INFINITY ? fminf(fmaxf(fmaxf(old, vn), 0x1p-126f), 0x1p126f) : vref;
    const float fo = vn == old ? 1.f : old / vn;
    if (__any_sync(kFull, fo != 1.f)) rescale_row(s, 8 * q, o, have_o, fo);
    return make_float3(mn, vn, f);
}

// The weights of a row over step b of a tile (64 tokens), 16 columns at a time,
// over the front of its scores: column pair i of P takes the place of score i,
// which has been read by then. Where a row's largest exponent in a chunk passes
// the lag, or may pass it times w, the row's maximum and reference are raised
// first. (Short loops: 32 columns at a time
// took 2 % longer, 64 in a row 15 %: eight warps run this code each at a place
// of its own, and fetching longer code costs more than its overlap gains.)
template <bool MASKED, bool WEIGH>
__device__ __forceinline__ void row_step(uint32_t s, uint32_t o, bool have_o, int b, const float2* scale, int page_log,
                                         bool real, bool joint, const View& view, RowState& st, Waiter& wait,
                                         uint32_t pv_done) {
    float inv = WEIGH ? reciprocal(st.vref) : 0.f;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const int col = 64 * b + 16 * q;
        const uint32_t seen = MASKED ? view.bits(col & ~31) >> (col & 31) : kFull;
        const float2 kv = scale[col >> page_log];
        uint32_t u[16];
        TmemLoad<16>::run(s + 16 * q, u);
        const bool some = !MASKED || (seen & 0xffffu);
        float most, sum, w = WEIGH ? value_factor(kv.y, some, st.vref, inv) : 1.f;
        uint32_t p[8];
        row_weights<MASKED, WEIGH>(u, seen, kv.x, w, st, most, sum, p);
        bool need = real && most > (WEIGH ? weight_limit(w) : kBias + kLag);
        if (__any_sync(kFull, need)) {
            // (a row before its first token may take its maximum early: of the step's
            // columns it is the same as behind the first one that it sees)
            need |= real && (joint || st.m == -INFINITY);
            if (have_o) {  // O is quiet once the step before is done; the one in
                           // front of that is, it came before these scores
                wait(pv_done, b ^ 1);
                tc_fence_after();
            }
            const float3 r = raise_row(s, o, have_o, q, b, MASKED ? view.bits(64 * b) : kFull,
                                       MASKED ? view.bits(64 * b + 32) : kFull, scale, page_log, st.c, need, st.m, st.vref);
            st.m = r.x;
            st.vref = r.y;
            st.l *= r.z;
            TmemLoad<16>::run(s + 16 * q, u);
            if (WEIGH) {
                inv = reciprocal(st.vref);
                w = value_factor(kv.y, some, st.vref, inv);
            }
            row_weights<MASKED, WEIGH>(u, seen, kv.x, w, st, most, sum, p);
        }
        st.l += sum;
        tmem_st8(s + 8 * q, reinterpret_cast<float*>(p));
    }
    tmem_wait_st();
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_rows_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ MapPair maps) {
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    Misc& ms = *reinterpret_cast<Misc*>(sm + kMisc);
    const int tid = threadIdx.x, lane = lane_id(), warp = __shfl_sync(kFull, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(smem_u32(&ms.k_full[i]), 1);
            mbar_init(smem_u32(&ms.k_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ms.v_full[i]), 1);
            mbar_init(smem_u32(&ms.v_empty[i]), 4);
            mbar_init(smem_u32(&ms.w_full[i]), 4);
            mbar_init(smem_u32(&ms.w_free[i]), 1);
            mbar_init(smem_u32(&ms.q_ready[i]), 4);
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&ms.s_full[i][b]), 1);
                mbar_init(smem_u32(&ms.p_full[i][b]), 4);
            }
            mbar_init(smem_u32(&ms.pv_done[i]), 1);
            mbar_init(smem_u32(&ms.o_full[i]), 1);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(smem_u32(&ms.sc_full[i]), 33);
        mbar_init(smem_u32(&ms.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(smem_u32(&ms.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;  // columns: S of half 0, S of half 1, O of half 0, O of half 1
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        const PagedRange r = paged_plan<RC, kSetup>(a, gridDim.x, blockIdx.x);
        if (lane == 0) ms.range = r;
    }
    __syncthreads();
    PagedWalk<RC, kSetup> walk(a, ms.range);
    const int G = (int)a.G.d, slots = kTile / a.page, page_log = 31 - __clz(a.page);
    Waiter wait;
    uint32_t it = 0;  // tiles of this CTA so far

    if (warp >= 12) {
        if (warp == 12) {
        // ------------------------------------------------------------ TMA --
        bool missing = false;
#pragma unroll 1
        for (; walk.live(); walk.next()) {
            const PagedUnit u = walk.u;
            const int j0 = walk.j0, j1 = walk.j1;
            const int32_t* row = a.seqs.table + walk.b * a.seqs.table_stride;
            auto fetch = [&](int j) -> int {  // this lane's page of a tile, -1 where no row sees it
                if (lane >= slots || j >= j1) return -1;
                const int slot = u.tile(j) * slots + lane, t0 = slot << page_log;
                if (t0 > u.p1 || (t0 + a.page <= u.lo_tok && t0 >= a.sinks)) return -1;
                const int id = row[slot];
                if (id >= 0 && id < a.num_pages) return id;
                missing = true;
                return -1;
            };
            int id = fetch(j0);
#pragma unroll 1
            for (int j = j0; j < j1; ++j, ++it) {
                const int next = fetch(j + 1);
                const uint32_t ks = it % kKStages, vs = it & 1, ring = it % kRing;
                const uint32_t k_full = smem_u32(&ms.k_full[ks]), v_full = smem_u32(&ms.v_full[vs]);
                const unsigned have = __ballot_sync(kFull, id >= 0);
                const uint32_t bytes = (uint32_t)__popc(have) * (uint32_t)a.page * 128u;
                const uint32_t off = (uint32_t)lane * (uint32_t)a.page * 128u;
                const int tile = id * a.Hkv + walk.h;
                wait(smem_u32(&ms.k_empty[ks]), ((it / kKStages) & 1) ^ 1);
                if (lane == 0) {
                    mbar_arrive_tx(k_full, bytes);
                    ms.ok[ring] = have;
                    mbar_arrive(smem_u32(&ms.sc_full[ring]));
                }
                __syncwarp();
                if (id >= 0) {
                    tma_tile(sb + kK + ks * 16384u + off, &maps.k, tile, k_full);
                    cp_async4(smem_u32(&ms.scale[ring][lane].x), a.ks + tile);
                    cp_async4(smem_u32(&ms.scale[ring][lane].y), a.vs + tile);
                }
                mbar_arrive_cp_async(smem_u32(&ms.sc_full[ring]));
                wait(smem_u32(&ms.v_empty[vs]), ((it >> 1) & 1) ^ 1);
                if (lane == 0) mbar_arrive_tx(v_full, bytes);
                __syncwarp();
                if (id >= 0) tma_tile(sb + kV + vs * 16384u + off, &maps.v, tile, v_full);
                id = next;
            }
        }
        if (missing) paged_report(a.seqs, kBadPage);
        // No copy is in flight at the end, not even after a wait that failed.
#pragma unroll 1
        for (uint32_t i = it < 3 ? 0 : it - 3; i < it; ++i)
            mbar_wait(smem_u32(&ms.k_full[i % kKStages]), (i / kKStages) & 1);
#pragma unroll 1
        for (uint32_t i = it < 2 ? 0 : it - 2; i < it; ++i) mbar_wait(smem_u32(&ms.v_full[i & 1]), (i >> 1) & 1);
        } else if (warp == 13) {
        // ------------------------------------------------------------ MMA --
        if (elect_one()) {
            // A step is 64 tokens: half of a tile. The scores of step i + 2 take the
            // place of the weights of step i, behind their P V (MMAs of a CTA run in
            // the order of issue), so that a half always has its next scores ready.
            constexpr uint32_t id_s = mma_idesc(128, 64, false, false), id_lo = id_s | kA_e5m2, id_o = mma_idesc(128, 128, false, true);
            uint32_t seg[2] = {0, 0}, np[2] = {0, 0};  // segments and weight steps of each half
#pragma unroll 1
            for (; walk.live(); walk.next()) {
                const int cnt = 2 * (walk.j1 - walk.j0);
                const int halves = walk.u.rows > 128 ? 2 : 1;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    if (hf < halves) wait(smem_u32(&ms.q_ready[hf]), seg[hf]++ & 1);
#pragma unroll 1
                for (int i = 0; i < cnt + 2; ++i) {
                    const uint32_t t = it + (i >> 1), tp = t - 1, b = i & 1;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        if (hf >= halves) continue;
                        if (i > 1) {
                            if (hf == 0 && b == 0) wait(smem_u32(&ms.w_full[tp & 1]), (tp >> 1) & 1);
                            wait(smem_u32(&ms.p_full[hf][b]), (np[hf] >> 1) & 1);
                            ++np[hf];
                            tc_fence_after();
                            const uint64_t vb = desc_sw128(sb + kV16 + (tp & 1) * 32768u + b * 8192u, 16384, 1024);
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // 16 tokens each
                                mma_f16_ts(tmem + 256 + hf * 128, tmem + hf * 128 + b * 64 + 8 * k, vb + 128 * k, id_o,
                                           i > 2 || k > 0);
                            mma_commit(smem_u32(&ms.pv_done[hf]));
                            if (i == cnt + 1) mma_commit(smem_u32(&ms.o_full[hf]));
                        }
                        if (i < cnt) {
                            if (hf == 0 && b == 0) {
                                wait(smem_u32(&ms.k_full[t % kKStages]), (t / kKStages) & 1);
                                tc_fence_after();
                            }
                            const uint64_t kb = desc_sw128(sb + kK + (t % kKStages) * 16384u + b * 8192u, 16, 1024);
                            const uint64_t qa = desc_sw128(sb + kQ + hf * 32768u, 16, 1024);
#pragma unroll
                            for (int k = 0; k < 8; ++k)  // 32 channels each; the pieces one after the other
                                mma_f8(tmem + hf * 128 + b * 64, qa + (k >> 2) * 1024 + 2 * (k & 3), kb + 2 * (k & 3),
                                       k < 4 ? id_s : id_lo, k > 0);
                            mma_commit(smem_u32(&ms.s_full[hf][b]));
                        }
                    }
                    if (i > 1 && b == 1) mma_commit(smem_u32(&ms.w_free[tp & 1]));
                    if (i < cnt && b == 1) mma_commit(smem_u32(&ms.k_empty[t % kKStages]));
                }
                it += cnt >> 1;
            }
            mma_commit(smem_u32(&ms.done));  // nor an MMA
            mbar_wait(smem_u32(&ms.done), 0);
        }
        __syncwarp();
        }
    } else if (warp >= 8) {
        // -------------------------------------------------- V to fp16 tiles --
        const int tok = tid - 256;  // token of the tile
        uint32_t seg[2] = {0, 0};
#pragma unroll 1
        for (; walk.live(); walk.next()) {
            const PagedUnit u = walk.u;
            const int j0 = walk.j0, j1 = walk.j1;
            wait(smem_u32(&ms.q_ready[0]), seg[0]++ & 1);  // the rows' NaN marks are clear
            if (u.rows > 128) wait(smem_u32(&ms.q_ready[1]), seg[1]++ & 1);
#pragma unroll 1
            for (int j = j0; j < j1; ++j, ++it) {
                const uint32_t buf = it & 1, ring = it % kRing;
                wait(smem_u32(&ms.sc_full[ring]), (it / kRing) & 1);
                wait(smem_u32(&ms.v_full[buf]), (it >> 1) & 1);
                wait(smem_u32(&ms.w_free[buf]), ((it >> 1) & 1) ^ 1);
                const int t = u.tile(j) * kTile + tok;
                const bool have = (ms.ok[ring] >> (tok >> page_log)) & 1u;
                const bool sink = t < a.sinks;
                const bool some = have && t <= u.p1 && (!a.window || sink || t >= u.p0 || t > u.p0 - a.window);
                const bool all = have && t <= u.p0 && (!a.window || sink || t > u.p1 - a.window);
                const uint8_t* src = sm + kV + buf * 16384 + tok * 128;
                uint8_t* dst = sm + kV16 + buf * 32768 + tok * 128;
#pragma unroll 2
                for (int c = 0; c < 8; ++c) {  // 16 channels each
                    uint4 q = *reinterpret_cast<const uint4*>(src + ((c ^ (tok & 7)) << 4));
                    uint32_t w[4] = {q.x, q.y, q.z, q.w};
                    if (!all) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (!some) w[k] = 0;
                            const uint32_t nan = __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            w[k] &= ~nan;
#pragma unroll 1
                            for (uint32_t left = nan & 0x01010101u; left; left &= left - 1) {
                                const int d = 16 * c + 4 * k + ((__ffs(left) - 1) >> 3);
#pragma unroll 1
                                for (int r = 0; r < u.rows; ++r) {
                                    const int gap = u.first_pos + (u.r0 + r) / G - t;
                                    if (gap >= 0 && (!a.window || sink || gap < a.window))
                                        atomicOr(&ms.nan[r][d >> 5], 1u << (d & 31));
                                }
                            }
                        }
                    }
                    uint8_t* half = dst + (c >> 2) * 16384;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4*>(half + (((2 * (c & 3) + k) ^ (tok & 7)) << 4)) =
                            make_uint4(e4m3x2_to_f16x2(w[2 * k] & 0xffffu), e4m3x2_to_f16x2(w[2 * k] >> 16),
                                       e4m3x2_to_f16x2(w[2 * k + 1] & 0xffffu), e4m3x2_to_f16x2(w[2 * k + 1] >> 16));
                }
                proxy_fence();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&ms.w_full[buf]));
                    mbar_arrive(smem_u32(&ms.v_empty[buf]));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ rows --
        const int hf = warp >> 2, r = tid;  // r: row of the unit
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + hf * 128, o_at = tmem + lanes + 256 + hf * 128;
        const uint32_t all_slots = (1u << slots) - 1u;
        const uint32_t pv_done = smem_u32(&ms.pv_done[hf]);
        uint32_t n = 0, seg = 0;  // weight tiles and segments of this half
#pragma unroll 1
        for (; walk.live(); walk.next()) {
            const PagedUnit u = walk.u;
            const int j0 = walk.j0, j1 = walk.j1;
            if (hf * 128 < u.rows) {
                const bool real = r < u.rows;
                const int rr = u.r0 + (real ? r : 0), qi = (int)fdiv((uint32_t)rr, a.G);
                const int64_t out_row = (int64_t)(u.row0 + qi) * a.Hq + walk.h * G + rr - qi * G;
                const int pos = real ? u.first_pos + qi : -1;
                // least and largest position of the warp's rows
                const int w0 = u.r0 + 32 * warp;
                const int wn = u.rows - 32 * warp < 32 ? u.rows - 32 * warp : 32;
                const int wp0 = u.first_pos + (int)fdiv((uint32_t)w0, a.G);
                const int wp1 = u.first_pos + (int)fdiv((uint32_t)(w0 + (wn > 0 ? wn : 1) - 1), a.G);
                const float c = write_rows(a, u, walk.h, 32 * warp, sm + kQ + hf * 32768, 32 * (warp & 3));
#pragma unroll
                for (int k = 0; k < 4; ++k) ms.nan[r][k] = 0u;
                proxy_fence();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.q_ready[hf]));
                RowState st{c, real ? -INFINITY : 0.f, 0.f, 0.f};
                bool joint = true;  // the warp's rows have seen the same tokens of the segment
#pragma unroll 1
                for (int j = j0; j < j1; ++j, ++it, ++n) {
                    const uint32_t ring = it % kRing;
                    // The scores first: a half without rows skips whole segments, and only
                    // with them is the ring's phase known to be this tile's or the one before.
                    wait(smem_u32(&ms.s_full[hf][0]), n & 1);
                    wait(smem_u32(&ms.sc_full[ring]), (it / kRing) & 1);
                    const int t0 = u.tile(j) * kTile;
                    const uint32_t ok = ms.ok[ring];
                    const float2* scale = ms.scale[ring];
                    const bool whole = ok == all_slots && t0 + kTile - 1 <= wp0 &&
                                       (!a.window || t0 > wp1 - a.window || t0 + kTile <= a.sinks);
                    const View view{pos - t0, a.window ? pos - t0 - a.window : -1, a.sinks - t0, ok, page_log};
                    // (scales are positive: their bits order like them)
                    const float vmax = __uint_as_float(__reduce_max_sync(
                        kFull, lane < slots && ((ok >> lane) & 1u) ? __float_as_uint(scale[lane].y) : 0u));
                    const float vmin = __uint_as_float(__reduce_min_sync(
                        kFull, lane < slots && ((ok >> lane) & 1u) ? __float_as_uint(scale[lane].y) : 0x7f800000u));
                    const bool one = whole && vmin == vmax;  // one v scale in the tile
                    joint &= whole;
#pragma unroll 1
                    for (int b = 0; b < 2; ++b) {
                        wait(smem_u32(&ms.s_full[hf][b]), n & 1);
                        tc_fence_after();
                        const bool have_o = j > j0 || b > 0;
                        const bool plain = one && __all_sync(kFull, !real || vmax == st.vref);
                        if (plain) row_step<false, false>(s_at + 64 * b, o_at, have_o, b, scale, page_log, real, joint, view, st, wait, pv_done);
                        else if (whole) row_step<false, true>(s_at + 64 * b, o_at, have_o, b, scale, page_log, real, joint, view, st, wait, pv_done);
                        else row_step<true, true>(s_at + 64 * b, o_at, have_o, b, scale, page_log, real, joint, view, st, wait, pv_done);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&ms.p_full[hf][b]));
                    }
                }
                wait(smem_u32(&ms.o_full[hf]), seg++ & 1);
                tc_fence_after();
                const bool complete = walk.complete();
                float* part = a.part + (2 * blockIdx.x + (walk.first ? 0 : 1)) * part_stride<RC>();
                const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
                __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + out_row * kD;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    float v[32];
                    tmem_ld<32>(o_at + 32 * q, v);
                    const uint32_t nan = ms.nan[r][q];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = (nan >> i) & 1u ? NAN : v[i] * inv * st.vref;
                    if (!real) continue;
                    if (complete) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = (uint32_t)f32_to_bf16_rn(v[i + 2 * k]) | ((uint32_t)f32_to_bf16_rn(v[i + 2 * k + 1]) << 16);
                            *reinterpret_cast<uint4*>(out + 32 * q + i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4*>(part + r * kD + 32 * q + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                }
                if (!complete && real) part[RC * kD + r] = st.m, part[RC * kD + RC + r] = st.l;
                tc_fence_before();
            } else {
                it += j1 - j0;
            }
        }
    }
    if (!wait.good) paged_report(a.seqs, kTimeout);
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace

size_t paged_rows_workspace() { return paged_workspace<RC>(device_sm_count()); }

cudaError_t launch_paged_rows(const PagedAttnArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};
    MapPair maps;
    cudaError_t e = make_pool_map(&maps.k, a.kc, a.num_pages * a.Hkv, a.page);
    if (e == cudaSuccess) e = make_pool_map(&maps.v, a.vc, a.num_pages * a.Hkv, a.page);
    if (e != cudaSuccess) return e;
    const int ctas = device_sm_count();
    e = launch_smem_pdl(paged_rows_kernel, ready, dim3(ctas), dim3(kThreads), kMisc + sizeof(Misc) + 1024, s, paged_lay_out(a, ctas), maps);
    if (e != cudaSuccess) return e;
    return launch_paged_join<RC>(paged_lay_out(a, ctas), ctas, s);
}

}  // namespace nsnq
