// Attention over the paged 8-bit cache for few query rows per kv-head: decode
// steps and drafted tokens; every row count for fp32 queries or outputs.
//
// The cache's e4m3 codes go to the tensor cores as they are: TMA brings a
// tile of 128 tokens of K and V into shared memory and tcgen05.mma
// (kind::f8f6f4) reads it there, so no thread touches a code and the kernel
// can run at the rate of the memory. What meets the codes has to be e4m3
// too: a query row and a column of weights are each split into pieces of 4
// significant bits,
//   x = sum_k 2^(-gk) e4m3(2^(gk) (x - pieces before)),  g = 5 or 6,
// and every piece is a column of its own. The scores of a tile are
//   S[token][piece, row] = K q^T   (M = 128 tokens, N = pieces x rows, K = 128 channels),
// lane t of TMEM holding token t; a thread adds its token's pieces, applies
// the page's scale, takes p = 2^(s - m), and writes w = p * v scale / 2^e in
// pieces, e the row's own (below); then
//   O[channel][piece, row] += V^T w   (M = 128 channels, K = 128 tokens).
// Two pieces hold a bf16 query exactly (8 bits; the row scaled to at most
// 256, elements below 2^-14 of that lose bits to an absolute 2^-24 of it);
// three hold weights to 2^-10, six hold fp32 queries and weights to 2^-24.
// Products of codes are exact in fp32, and fp32 is what TMEM accumulates.
// (The alternative, widening K and V to 16 bits for kind::f16, would write and
// read every tile once more through shared memory: 64 KB more for the 32 KB
// that arrive, next to 32 KB that the MMAs read now.)
//
// The running maximum m of a row may lag by 2^kLag, so that a tile seldom
// needs it raised: a vote of the 128 token threads per tile decides; sums of
// p stay per thread until the segment ends. A second maximum per row, with the
// same lag, is that of log2 p + log2 v scale; its distance from the first one, in
// whole powers of two, is the e of w, so that w spans the pieces' range whatever
// the scales are. The bias 2^kBias keeps the smallest piece at 2^-23 of the row's
// largest w. Where every row's 2^e is the token's v scale (equal scales, powers of
// two), w is p. No bit of a row depends on what it does not see: the unit's rows
// raise their maxima together while all of them have seen the same tokens (rows of
// one position, or whole tiles so far), from then on each by itself. (A raise holds
// up the tile; rows that raise one by one do so in a fifth to a third more tiles.)
//
// What bounds it: memory for up to 4 rows (16 sequences x 32k tokens, 8
// kv-heads, 4 query heads each: 165 to 169 us, 6.4 to 6.5 TB/s, 97 to 99 % of the
// measured copy rate); one 131k sequence 54 us (5.0 TB/s: start, join and the longer
// waits of single pages weigh in). With 8 and 16 rows the token warps' work does:
// 64 sequences under a 2048 window, 8 heads 64 us (4.3 TB/s), 13 x 4 drafted rows
// over ~6k tokens, 4 heads 53 us (3.0 TB/s). A lag of 2^3 instead of 2^5 raised
// maxima in half of those tiles (69 us). One-CUDA-core-row-per-block attention,
// the first version, took 6461 us for the 16 x 32k batch.
#include <math.h>

#include "attn_split.cuh"
#include "paged_join.cuh"

namespace nsnq {

namespace {

constexpr int kThreads = 192;  // warps 0-3: tokens / channels; 4: TMA; 5: MMA issue
constexpr float kLag = 5.f, kBias = 2.f;  // weights stay below 2^7 (1 + 2^-20)
// Bits between the pieces of a weight. A piece rounds its value to within 2^(k - 4)
// below 2^(k + 1), so that with 5 the next piece stays below the same bound. With 6
// it doubles: of a weight from 2^6 to 2^7 the third piece may be held at 448 where it
// would be 512, 2^-12 of the weight besides fp16's 2^-11.
constexpr int shift_of(int pieces) { return pieces <= 3 ? 6 : 5; }
constexpr int kMaxSlots = 8;   // pages per tile (page_size 16)
constexpr int kMaxRows = 16;   // of a unit
// Tiles that a unit's queries and epilogue cost (1, 2, 3: 13 x 4 rows 57.0, 55.3,
// 55.1 us; 64 windows 65.4, 65.2, 64.3).
constexpr int kSetup = 3;

constexpr int pad16(int n) { return (n + 15) / 16 * 16; }
constexpr int pow2_at_least(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256; }  // TMEM columns

// RC rows per unit, QP pieces of a query, PP pieces of a weight.
template <int RC, int QP, int PP>
struct Shape {
    static constexpr int N1 = pad16(RC * QP), N2 = pad16(RC * PP);
    static constexpr int kStages = RC <= 8 && PP <= 3 ? 3 : 2;  // of 32 KB; two CTAs share an SM
    static constexpr int kTmem = pow2_at_least(2 * N1 + N2);
    // shared memory, from a 1024-aligned base
    static constexpr uint32_t kK = 0, kV = kK + kStages * 16384, kQ = kV + kStages * 16384,
                              kP = kQ + N1 * 128, kMisc = kP + 2 * N2 * 128;
};

struct Misc {
    uint64_t full[3], empty[3], s_full[2], s_free[2], p_full[2], p_free[2], q_ready, done;
    uint32_t tmem;
    PagedRange range;
    uint32_t ok[3];               // stage: pages of the tile that were loaded
    float ks[3][kMaxSlots], vs[3][kMaxSlots];
    float qs[kMaxRows];                 // row: score scale (softmax scale, log2 e, query scale)
    int pos[kMaxRows];                  // row: token position
    // each warp's own copy, for row: score scale, bias - maximum; 2^-e and -e, w = p * v scale * 2^-e
    float2 cb[4][kMaxRows];
    alignas(16) float rv[4][kMaxRows];
    alignas(16) float lrv[4][kMaxRows];
    float2 factor[4][kMaxRows];         // as a row's maxima rise: of its sum of weights, of its outputs
    float2 red[4][kMaxRows];            // a warp's tokens: largest score, largest score + log2 v scale
    float sums[4][kMaxRows];
    uint32_t nan[kMaxRows][4];          // row: channels that a NaN code of a partly seen tile reaches
};

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_rest(uint32_t h, uint32_t c) {  // (h - c) * 2^6, exact
    uint32_t r;
    asm("{.reg .b32 d;\n\tsub.f16x2 d, %1, %2;\n\tmul.f16x2 %0, d, %3;}" : "=r"(r) : "r"(h), "r"(c), "r"(0x54005400u));
    return r;
}

// The pieces of two weights (rows r and r + 1): out[k] holds piece k's two codes.
template <int PP>
__device__ __forceinline__ void weight_pieces(float w0, float w1, uint32_t (&out)[PP]) {
    if constexpr (PP <= 3) {  // 11 bits of fp16 are enough to start from
        uint32_t h = f16x2(w0, w1);
#pragma unroll
        for (int k = 0; k < PP; ++k) {
            out[k] = e4m3x2_of_f16x2(h);
            if (k + 1 < PP) h = f16x2_rest(h, e4m3x2_to_f16x2(out[k]));
        }
    } else {
#pragma unroll
        for (int k = 0; k < PP; ++k) {
            out[k] = e4m3x2(w0, w1);
            const uint32_t h = e4m3x2_to_f16x2(out[k]);
            w0 = (w0 - f16_lo(h)) * (float)(1 << shift_of(PP));
            w1 = (w1 - f16_hi(h)) * (float)(1 << shift_of(PP));
        }
    }
}

// The weights of a token from their exponents z, added to the rows' sums l, and
// the pieces of what meets the values. ONE: for every token of the warp that is
// the weight itself; else only where vs = 0.
template <int RC, int PP, bool ONE>
__device__ __forceinline__ void weigh(const float* rv, const float (&z)[RC], float vs, float (&l)[RC],
                                      uint32_t (&word)[pad16(RC * PP) / 4]) {
#pragma unroll
    for (int i = 0; i < pad16(RC * PP) / 4; ++i) word[i] = 0;
#pragma unroll
    for (int r = 0; r < RC; r += 2) {
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[i] = exp2_approx(z[r + i]);
            l[r + i] += w[i];
            // (2^-e first: finite next to the largest scale, and a weight of 0 stays 0)
            if (!ONE) w[i] = vs != 0.f ? w[i] * rv[r + i] * vs : w[i];
        }
        uint32_t c[PP];
        weight_pieces<PP>(w[0], w[1], c);
#pragma unroll
        for (int k = 0; k < PP; ++k) word[(k * RC + r) / 4] |= c[k] << (((k * RC + r) & 2) * 8);
    }
}

__device__ __forceinline__ void bar_tokens() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool any_token(bool v) {  // vote of the 128 token threads
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Scores of this thread's token: the pieces of each row added up, under the
// token's k scale (not yet the row's).
template <int RC, int QP>
__device__ __forceinline__ void row_scores(uint32_t s, float ks, float (&y)[RC]) {
    constexpr int W = RC * QP % 32 == 0 ? 32 : RC * QP % 16 == 0 ? 16 : 8;  // columns a load
#pragma unroll
    for (int c0 = 0; c0 < RC * QP; c0 += W) {
        float v[W];
        tmem_ld<W>(s + c0, v);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int k = (c0 + i) / RC, r = (c0 + i) % RC;
            y[r] = k == 0 ? v[i] : fmaf(v[i], 1.f / (float)(1ull << (5 * k)), y[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < RC; ++r) y[r] *= ks;
}

__device__ __forceinline__ float warp_max_f32(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float power_of_two(float e) {  // of a whole number e from -126 to 127
    return __uint_as_float((uint32_t)((int)e + 127) << 23);
}

// The rows' state of a segment, kept by every warp alike: lane l has row l % RC's
// maximum m (log2 units) and exponent -e.
struct RowState {
    float m, lrv;
    float v_one;    // the v scale under which every row's w is p (0: none)
    float lrv_top;  // the largest -e of a row that has seen a token
};
template <int RC>
__device__ __forceinline__ RowState first_state(Misc& ms, int warp, int rows) {
    const int r = lane_id() % RC;
    ms.cb[warp][r] = make_float2(ms.qs[r], r < rows ? INFINITY : kBias);
    ms.rv[warp][r] = 1.f;
    ms.lrv[warp][r] = 0.f;
    __syncwarp();
    return {r < rows ? -INFINITY : 0.f, 0.f, 0.f, 0.f};
}
// Rows' maxima raised to the tile's (ms.red), all of them or (joint: false) where
// the tile passes a lag. The e is
// the whole number below the distance of the maxima (or at most 1/16 above it, for
// the rounding of their sum), so that the largest w is between 2^kBias and twice
// that; its bounds keep p * 2^-e finite.
template <int RC>
__device__ __forceinline__ void raise_maxima(Misc& ms, int warp, bool joint, RowState& st) {
    const int r = lane_id() % RC;
    const float top = fmaxf(fmaxf(ms.red[0][r].x, ms.red[1][r].x), fmaxf(ms.red[2][r].x, ms.red[3][r].x));
    const float top_w = fmaxf(fmaxf(ms.red[0][r].y, ms.red[1][r].y), fmaxf(ms.red[2][r].y, ms.red[3][r].y));
    const bool need = (joint && top > -INFINITY) || top - st.m > kLag || top_w - st.m + st.lrv > kLag;
    const float mn = need ? fmaxf(st.m, top) : st.m, e0 = -st.lrv;
    const float e = need ? fminf(fmaxf(floorf(fmaxf(st.m + e0, top_w) - mn + 0.0625f), -118.f), 126.f) : e0;
    const float down = st.m == mn ? 0.f : st.m - mn;
    ms.factor[warp][r] = make_float2(exp2_approx(down), exp2_approx(down + (e0 - e)));
    st.m = mn;
    st.lrv = -e;
    ms.cb[warp][r].y = kBias - mn;
    ms.rv[warp][r] = power_of_two(st.lrv);
    ms.lrv[warp][r] = st.lrv;
    __syncwarp();
}
// The same for every row: v_one and lrv_top.
template <int RC>
__device__ __forceinline__ void sum_up(RowState& st, int rows) {
    const bool seen = lane_id() % RC < rows && st.m > -INFINITY;
    const unsigned who = __ballot_sync(kFull, seen);
    const float first = __shfl_sync(kFull, st.lrv, who ? __ffs(who) - 1 : 0);
    st.v_one = __all_sync(kFull, !seen || st.lrv == first) ? power_of_two(-first) : 0.f;
    st.lrv_top = warp_max_f32(seen ? st.lrv : -INFINITY);
}

template <int RC, int QP, typename QT>
__device__ __forceinline__ void write_queries(const PagedAttnArgs& a, const PagedUnit& u, int h, uint8_t* q_sm,
                                              Misc& ms) {
    const int G = (int)a.G.d;
    const int lane = lane_id(), warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int r = warp; r < RC; r += 4) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        int pos = -1;
        if (r < u.rows) {
            const int rr = u.r0 + r, i = (int)fdiv((uint32_t)rr, a.G), hq = h * G + rr - i * G;
            load4(reinterpret_cast<const QT*>(a.q) + (int64_t)(u.row0 + i) * a.q_st + (int64_t)hq * a.q_sh + 4 * lane, x);
            pos = u.first_pos + i;
        }
        float top = 0.f;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            top = fmaxf(top, fabsf(x[k]));
            bad |= !isfinite(x[k]);
        }
        top = warp_max(top);
        bad = __any_sync(kFull, bad);
        // the least e >= -126 with top <= 256 * 2^e
        const uint32_t bits = __float_as_uint(top);
        int e = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) ? 7 : 8);
        e = bad ? 0 : (e < -126 ? -126 : e);
        const float up = __uint_as_float((uint32_t)(127 - e) << 23), down = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] *= up;
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const int n = k * RC + r;
            uint32_t c0 = e4m3x2(x[0], x[1]), c1 = e4m3x2(x[2], x[3]);
            const uint32_t h0 = e4m3x2_to_f16x2(c0), h1 = e4m3x2_to_f16x2(c1);
            x[0] = (x[0] - f16_lo(h0)) * 32.f;
            x[1] = (x[1] - f16_hi(h0)) * 32.f;
            x[2] = (x[2] - f16_lo(h1)) * 32.f;
            x[3] = (x[3] - f16_hi(h1)) * 32.f;
            const uint32_t word = bad ? 0x7f7f7f7fu : (c0 | (c1 << 16));
            *reinterpret_cast<uint32_t*>(q_sm + n * 128 + (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4) = word;
        }
        if (lane == 0) {
            ms.qs[r] = a.scale_log2 * down;
            ms.pos[r] = pos;
#pragma unroll
            for (int k = 0; k < 4; ++k) ms.nan[r][k] = 0u;
        }
    }
}

template <int RC, int QP, int PP, typename QT>
__global__ void __launch_bounds__(kThreads, 2)
    paged_cols_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ MapPair maps) {
    using Sh = Shape<RC, QP, PP>;
    constexpr int N1 = Sh::N1, N2 = Sh::N2, ST = Sh::kStages;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    Misc& ms = *reinterpret_cast<Misc*>(sm + Sh::kMisc);
    const int tid = threadIdx.x, lane = lane_id(), warp = __shfl_sync(kFull, tid >> 5, 0);

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < ST; ++i) {
            mbar_init(smem_u32(&ms.full[i]), 33);
            mbar_init(smem_u32(&ms.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ms.s_full[i]), 1);
            mbar_init(smem_u32(&ms.s_free[i]), 4);
            mbar_init(smem_u32(&ms.p_full[i]), 4);
            mbar_init(smem_u32(&ms.p_free[i]), 1);
        }
        mbar_init(smem_u32(&ms.q_ready), 4);
        mbar_init(smem_u32(&ms.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(smem_u32(&ms.tmem), Sh::kTmem);
#pragma unroll 1
    for (int i = tid; i < (N1 * 128 + 2 * N2 * 128) / 16; i += kThreads)  // padding columns stay zero
        reinterpret_cast<uint4*>(sm + Sh::kQ)[i] = make_uint4(0, 0, 0, 0);
    // Stale rows of a partly loaded tile must be finite before the first use.
#pragma unroll 1
    for (int i = tid; i < ST * 16384 / 16; i += kThreads)
        reinterpret_cast<uint4*>(sm + Sh::kV)[i] = make_uint4(0, 0, 0, 0);
    proxy_fence();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        const PagedRange r = paged_plan<RC, kSetup>(a, gridDim.x, blockIdx.x);
        if (lane == 0) ms.range = r;
    }
    __syncthreads();
    PagedWalk<RC, kSetup> walk(a, ms.range);
    const int G = (int)a.G.d;
    const int slots = kTile / a.page;
    Waiter wait;
    uint32_t it = 0;  // tiles of this CTA so far

    if (warp == 4) {
        // ------------------------------------------------------------ TMA --
        const int page_log = 31 - __clz(a.page);
        bool missing = false;
#pragma unroll 1
        for (; walk.live(); walk.next()) {
            const PagedUnit u = walk.u;
            const int j0 = walk.j0, j1 = walk.j1;
            const int32_t* row = a.seqs.table + walk.b * a.seqs.table_stride;
            // this lane's page of a tile, -1 where no row sees it
            auto fetch = [&](int j) -> int {
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
                const uint32_t st = it % ST, full = smem_u32(&ms.full[st]);
                wait(smem_u32(&ms.empty[st]), ((it / ST) & 1) ^ 1);
                const unsigned have = __ballot_sync(kFull, id >= 0);
                if (lane == 0) {
                    ms.ok[st] = have;
                    mbar_arrive_tx(full, (uint32_t)__popc(have) * 2u * (uint32_t)a.page * 128u);
                }
                __syncwarp();
                if (id >= 0) {
                    const int tile = id * a.Hkv + walk.h;
                    const uint32_t off = st * 16384u + (uint32_t)lane * (uint32_t)a.page * 128u;
                    tma_tile(sb + Sh::kK + off, &maps.k, tile, full);
                    tma_tile(sb + Sh::kV + off, &maps.v, tile, full);
                    cp_async4(smem_u32(&ms.ks[st][lane]), a.ks + tile);
                    cp_async4(smem_u32(&ms.vs[st][lane]), a.vs + tile);
                }
                mbar_arrive_cp_async(full);
                id = next;
            }
        }
        if (missing) paged_report(a.seqs, kBadPage);
        // No copy is in flight at the end, not even after a wait that failed.
#pragma unroll 1
        for (uint32_t i = it < ST ? 0 : it - ST; i < it; ++i) mbar_wait(smem_u32(&ms.full[i % ST]), (i / ST) & 1);
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA --
        if (elect_one()) {
            constexpr uint32_t id_s = mma_idesc(128, N1, false, false);  // K rows x query columns
            constexpr uint32_t id_o = mma_idesc(128, N2, true, true);    // V^T (channels) x weights
            uint32_t seg = 0;
#pragma unroll 1
            for (; walk.live(); walk.next(), ++seg) {
                const int cnt = walk.j1 - walk.j0;
                wait(smem_u32(&ms.q_ready), seg & 1);
#pragma unroll 1
                for (int i = 0; i <= cnt; ++i) {
                    if (i < cnt) {
                        const uint32_t t = it + i, st = t % ST;
                        wait(smem_u32(&ms.full[st]), (t / ST) & 1);
                        wait(smem_u32(&ms.s_free[t & 1]), ((t >> 1) & 1) ^ 1);
                        tc_fence_after();
                        const uint64_t ka = desc_sw128(sb + Sh::kK + st * 16384u, 16, 1024);
                        const uint64_t qb = desc_sw128(sb + Sh::kQ, 16, 1024);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 channels each
                            mma_f8(tmem + (t & 1) * N1, ka + 2 * k, qb + 2 * k, id_s, k > 0);
                        mma_commit(smem_u32(&ms.s_full[t & 1]));
                    }
                    if (i > 0) {
                        const uint32_t t = it + i - 1, st = t % ST;
                        wait(smem_u32(&ms.p_full[t & 1]), (t >> 1) & 1);
                        tc_fence_after();
                        const uint64_t va = desc_sw128(sb + Sh::kV + st * 16384u, 16384, 1024);
                        const uint64_t pb = desc_plain(sb + Sh::kP + (t & 1) * N2 * 128, 128, 2048);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 tokens each
                            mma_f8(tmem + 2 * N1, va + 256 * k, pb + 32 * k, id_o, i > 1 || k > 0);
                        mma_commit(smem_u32(&ms.p_free[t & 1]));
                        mma_commit(smem_u32(&ms.empty[st]));
                    }
                }
                it += cnt;
            }
            mma_commit(smem_u32(&ms.done));  // nor an MMA
            mbar_wait(smem_u32(&ms.done), 0);
        }
        __syncwarp();
    } else {
        // --------------------------------------------- tokens, then channels --
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const int page_log = 31 - __clz(a.page), slot = tid >> page_log;
        const uint32_t all_slots = (1u << slots) - 1u;
#pragma unroll 1
        for (; walk.live(); walk.next()) {
            const PagedUnit u = walk.u;
            const int j0 = walk.j0, j1 = walk.j1;
            const uint32_t real = (1u << u.rows) - 1u;
            bar_tokens();  // the segment before is done with the row data
            write_queries<RC, QP, QT>(a, u, walk.h, sm + Sh::kQ, ms);
            proxy_fence();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.q_ready));
            bar_tokens();
            RowState state = first_state<RC>(ms, warp, u.rows);
            const float2* row_cb = ms.cb[warp];
            bool joint = true;  // the rows have seen the same tokens of the segment
            float l[RC];
#pragma unroll
            for (int r = 0; r < RC; ++r) l[r] = 0.f;
#pragma unroll 1
            for (int j = j0; j < j1; ++j, ++it) {
                const uint32_t buf = it & 1, st = it % ST;
                wait(smem_u32(&ms.s_full[buf]), (it >> 1) & 1);
                wait(smem_u32(&ms.full[st]), (it / ST) & 1);
                tc_fence_after();
                const int tile = u.tile(j), tok = tile * kTile + tid;
                const uint32_t have = ms.ok[st];
                const bool whole = have == all_slots && tile * kTile + kTile - 1 <= u.p0 &&
                                   (!a.window || tile * kTile > u.p1 - a.window || tile * kTile + kTile <= a.sinks);
                joint &= whole || u.p0 == u.p1;
                const float ks = ms.ks[st][slot], vs = ms.vs[st][slot];
                uint32_t vis = real;
                if (!whole) {
                    vis = 0;
                    if ((have >> slot) & 1u) {
                        const int back = a.window && tok >= a.sinks ? a.window : 0x7fffffff;
#pragma unroll
                        for (int r = 0; r < RC; ++r) {
                            const int gap = ms.pos[r] - tok;
                            vis |= (gap >= 0 && gap < back ? 1u : 0u) << r;
                        }
                        vis &= real;
                    }
                }
                float z[RC];  // exponents of the weights: score - maximum + bias, log2 units
                row_scores<RC, QP>(lanes + buf * N1, ks, z);
#pragma unroll
                for (int r = 0; r < RC; ++r) {
                    const float2 cb = row_cb[r];
                    z[r] = fmaf(z[r], cb.x, cb.y);
                }
                if (vis != (1u << RC) - 1u) {
#pragma unroll
                    for (int r = 0; r < RC; ++r) z[r] = (vis >> r) & 1u ? z[r] : -INFINITY;
                }
                float most = z[0];
#pragma unroll
                for (int r = 1; r < RC; ++r) most = fmaxf(most, z[r]);
                bool over = most > kBias + kLag;
                if (vis != 0 && vs != state.v_one) {  // some row's w may be too large where its p is not
                    const float lvs = __log2f(vs);
                    if (most + lvs + state.lrv_top > kBias + kLag) {
#pragma unroll
                        for (int r = 0; r < RC; ++r) over |= z[r] + (lvs + ms.lrv[warp][r]) > kBias + kLag;
                    }
                }
                if (any_token(over)) {
                    // raise the maxima: per row over the tile's tokens
                    const float lvs = __log2f(vs), vs0 = __shfl_sync(kFull, vs, 0);
                    const bool alike = __all_sync(kFull, vis == 0 || vs == vs0);
                    row_scores<RC, QP>(lanes + buf * N1, ks, z);
#pragma unroll
                    for (int r = 0; r < RC; ++r) {
                        const float x = (vis >> r) & 1u ? z[r] * row_cb[r].x : -INFINITY, top = warp_max_f32(x);
                        const float top_w = alike ? top + lvs : warp_max_f32((vis >> r) & 1u ? x + lvs : -INFINITY);
                        if (lane == 0) ms.red[warp][r] = make_float2(top, top_w);
                    }
                    bar_tokens();  // (red is written again behind the next vote at the earliest)
                    raise_maxima<RC>(ms, warp, joint, state);
                    float f[RC];
#pragma unroll
                    for (int r = 0; r < RC; ++r) {
                        const float2 cb = row_cb[r], by = ms.factor[warp][r];
                        l[r] *= by.x;
                        f[r] = by.y;
                        z[r] = (vis >> r) & 1u ? fmaf(z[r], cb.x, cb.y) : -INFINITY;
                    }
                    if (j > j0) {
                        wait(smem_u32(&ms.p_free[buf ^ 1]), ((it - 1) >> 1) & 1);
                        tc_fence_after();
#pragma unroll
                        for (int c0 = 0; c0 < RC * PP; c0 += 8) {
                            float v[8];
                            tmem_ld<8>(lanes + 2 * N1 + c0, v);
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[i] *= f[(c0 + i) % RC];
                            tmem_st8(lanes + 2 * N1 + c0, v);
                        }
                        tmem_wait_st();
                    }
                    sum_up<RC>(state, u.rows);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.s_free[buf]));
                const bool one = vis == 0 || vs == state.v_one;  // w is p
                uint32_t word[N2 / 4];
                if (__all_sync(kFull, one)) weigh<RC, PP, true>(ms.rv[warp], z, 0.f, l, word);
                else weigh<RC, PP, false>(ms.rv[warp], z, one ? 0.f : vs, l, word);
                wait(smem_u32(&ms.p_free[buf]), ((it >> 1) & 1) ^ 1);
#pragma unroll
                for (int i = 0; i < N2 / 16; ++i)
                    *reinterpret_cast<uint4*>(sm + Sh::kP + buf * N2 * 128 + i * 2048 + tid * 16) =
                        make_uint4(word[4 * i], word[4 * i + 1], word[4 * i + 2], word[4 * i + 3]);
                if (!whole && vis != real) {
                    // a token that some row does not see: its values must not
                    // meet that row's zero weight as NaN
                    uint8_t* vrow = sm + Sh::kV + st * 16384 + tid * 128;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const int pc = (i + lane) & 7;  // spreads the lanes over the banks
                        uint4* at = reinterpret_cast<uint4*>(vrow + pc * 16);
                        if (!vis) {
                            *at = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        uint32_t c[4] = {at->x, at->y, at->z, at->w};
                        uint32_t any = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t nan = __vcmpeq4(c[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            any |= nan;
                            c[k] &= ~nan;
                            const int d0 = ((pc ^ (tid & 7)) << 4) + 4 * k;
#pragma unroll 1
                            for (uint32_t left = nan & 0x01010101u; left; left &= left - 1)
#pragma unroll 1
                                for (uint32_t seen = vis; seen; seen &= seen - 1) {
                                    const int d = d0 + ((__ffs(left) - 1) >> 3);
                                    atomicOr(&ms.nan[__ffs(seen) - 1][d >> 5], 1u << (d & 31));
                                }
                        }
                        if (any) *at = make_uint4(c[0], c[1], c[2], c[3]);
                    }
                }
                proxy_fence();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.p_full[buf]));
            }
            // ---- the segment's rows: sums over the tokens, channels from TMEM ----
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                const float s = warp_sum(l[r]);
                if (lane == 0) ms.sums[warp][r] = s;
            }
            wait(smem_u32(&ms.p_free[(it - 1) & 1]), ((it - 1) >> 1) & 1);
            tc_fence_after();
            bar_tokens();
            float o[RC];
#pragma unroll
            for (int r = 0; r < RC; ++r) o[r] = 0.f;
#pragma unroll
            for (int c0 = 0; c0 < RC * PP; c0 += 8) {
                float v[8];
                tmem_ld<8>(lanes + 2 * N1 + c0, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int k = (c0 + i) / RC, r = (c0 + i) % RC;
                    if (k < PP) o[r] = k == 0 ? v[i] : fmaf(v[i], 1.f / (float)(1ull << (shift_of(PP) * k)), o[r]);
                }
            }
            tc_fence_before();
            const bool complete = walk.complete();
            float* part = a.part + (int64_t)(2 * blockIdx.x + (walk.first ? 0 : 1)) * part_stride<RC>();
            const int lr = lane % RC;  // this lane's row
            const float sum = ms.sums[0][lr] + ms.sums[1][lr] + ms.sums[2][lr] + ms.sums[3][lr];
            const float inv = sum == 0.f ? 0.f : 1.f / sum, vref = power_of_two(-state.lrv);
            if (!complete && tid < u.rows) part[RC * kD + tid] = state.m, part[RC * kD + RC + tid] = sum;
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                if (r >= u.rows) continue;
                float v = o[r] * __shfl_sync(kFull, inv, r) * __shfl_sync(kFull, vref, r);
                if ((ms.nan[r][tid >> 5] >> (tid & 31)) & 1u) v = NAN;
                if (!complete) {
                    part[r * kD + tid] = v;
                    continue;
                }
                const int rr = u.r0 + r, i = (int)fdiv((uint32_t)rr, a.G);
                store_out(a, (int64_t)(u.row0 + i) * a.Hq + walk.h * G + rr - i * G, tid, v);
            }
        }
    }
    if (!wait.good) paged_report(a.seqs, kTimeout);
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, Sh::kTmem);
}

template <int RC, int QP, int PP, typename QT>
cudaError_t launch_cols(const PagedAttnArgs& a, cudaStream_t s) {
    using Sh = Shape<RC, QP, PP>;
    static std::atomic<unsigned long long> ready{0};
    MapPair maps;
    cudaError_t e = make_pool_map(&maps.k, a.kc, a.num_pages * a.Hkv, a.page);
    if (e == cudaSuccess) e = make_pool_map(&maps.v, a.vc, a.num_pages * a.Hkv, a.page);
    if (e != cudaSuccess) return e;
    const int ctas = 2 * device_sm_count();
    e = launch_smem_pdl(paged_cols_kernel<RC, QP, PP, QT>, ready, dim3(ctas), dim3(kThreads),
                        Sh::kMisc + sizeof(Misc) + 1024, s, paged_lay_out(a, ctas), maps);
    if (e != cudaSuccess) return e;
    return launch_paged_join<RC>(paged_lay_out(a, ctas), ctas, s);
}

// Rows of a unit: the least power of two that holds a sequence's rows of one
// kv-head; at most 16, and 8 where fp32 takes six pieces of everything.
int unit_rows(int64_t pairs, bool f32) {
    if (pairs <= 4) return 4;
    if (pairs <= 8 || f32) return 8;
    return 16;
}

}  // namespace

size_t paged_attn_workspace(int64_t n_rows, int, int Hq, int Hkv, int64_t max_rows) {
    const int64_t rows = max_rows < n_rows ? max_rows : n_rows;
    const int rc = unit_rows(rows * (Hq / Hkv), false);
    const int ctas = 2 * device_sm_count();
    const size_t cols = rc <= 8 ? paged_workspace<8>(ctas) : paged_workspace<16>(ctas);
    const size_t whole = paged_rows_workspace();
    return rows * (Hq / Hkv) > kMaxRows && whole > cols ? whole : cols;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
    const int64_t rows = a.max_rows < a.seqs.n_rows ? a.max_rows : a.seqs.n_rows;
    const bool f32 = !a.q_bf16 || !a.out_bf16;
    const int rc = unit_rows(rows * (a.Hq / a.Hkv), f32);
    if (f32) {
        if (a.q_bf16)
            return rc == 4 ? launch_cols<4, 2, 6, __nv_bfloat16>(a, s) : launch_cols<8, 2, 6, __nv_bfloat16>(a, s);
        return rc == 4 ? launch_cols<4, 6, 6, float>(a, s) : launch_cols<8, 6, 6, float>(a, s);
    }
    // More rows than a unit here takes go to 256-row units on their own kernel. A
    // variant of this one for 32 rows took as long or longer: 8 sequences of 8k
    // tokens, 20 and 32 rows per kv-head, 84.5 and 92.1 us against 85.5 and 87.8;
    // 40 of 500 tokens, 32 rows, 71 against 60 us.
    if (rows * (a.Hq / a.Hkv) > kMaxRows) return launch_paged_rows(a, s);
    switch (rc) {
        case 4: return launch_cols<4, 2, 3, __nv_bfloat16>(a, s);
        case 8: return launch_cols<8, 2, 3, __nv_bfloat16>(a, s);
        default: return launch_cols<16, 2, 3, __nv_bfloat16>(a, s);
    }
}

}  // namespace nsnq
