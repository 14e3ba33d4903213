// Append to the paged 8-bit cache: new keys and values, the keys (and
// queries) rotated to their positions, stored in e4m3 under one power-of-two
// scale per (page, head).
//
// x -> code = e4m3(x / 2^e), e the least exponent with every |x| of the
// (page, head) <= 448 * 2^e. One block owns a page for its heads of K or V, so
// the page's scale, the codes of its new tokens and, where the scale grows,
// the renewed codes of its older tokens have a single writer and no atomics.
//
// Codes and scales are those of the fp64 rotation, decided in fp32: angles are
// reduced in fp64, cos and sin rounded to fp32, and a rotated value is then
// off by at most 2^-21.8 (|x| + |y|) of its pair (x, y): the roundings of the angle,
// of cos or sin, of a product and of the sum. Where a code or scale would change
// within twice that, it is decided again from an fp64 rotation (about one code in
// 10^5). The cos and sin of a page's rows are computed once
// per block, in shared memory, and serve all its heads. Queries are not decisions:
// bf16 ones are rounded from the fp32 rotation (deciding again where that is not
// sure of the nearest bf16 took 257 us instead of 181 below, for one bit in 3 *
// 10^4 values), fp32 ones from one in two words (21 -> 23 us, 5 x ~580 rows).
//
// What bounds it: memory, in the end (a row is read once and written once; the
// next heads' rows are copied to shared memory ahead by cp.async). A prompt of
// 8 x 4096 tokens, 8 kv-heads and 32 query heads, bf16 takes 183 us: 738 MB at
// 4.0 TB/s (61 % of the measured copy rate). fp64 throughout took 498 us, fp32
// with one head's rows in flight 311, with the next head's in registers 196.
//
#include <math.h>

#include "paged.cuh"

namespace nsnq {

namespace {

// A row is 8 lanes, lane l holding channels [8l, 8l + 8) of both halves (the
// rotation's pairs). A thread takes kPasses rows of a page.
template <int PAGE>
struct AppShape {
    static constexpr int kPasses = PAGE == 16 ? 1 : 2;
    static constexpr int kThreads = PAGE * 8 / kPasses;
};
// Heads whose rows a block has on their way or at hand.
template <typename XT>
constexpr int app_ahead() { return sizeof(XT) == 2 ? 3 : 2; }
constexpr float kErr = 0x1p-20f;  // of |lo| + |hi|, rotated: >= 2^-21.8 (|x| + |y|) and as much again

// The least e >= -126 with a <= 448 * 2^e, for finite a >= 0:
// a = f * 2^k with 1 <= f < 2, and 448 = 1.75 * 2^8.
__device__ __forceinline__ int cover_exponent(double a) {
    if (!(a > 0.0)) return -126;
    const long long u = __double_as_longlong(a);
    const int k = (int)(u >> 52) - 1023;  // every fp32 product and sum is normal in fp64
    const int e = (u & 0xfffffffffffffll) > 0xc000000000000ll ? k - 7 : k - 8;
    return e < -126 ? -126 : e;
}
__device__ __forceinline__ double exp2i(int e) {
    return __longlong_as_double((long long)(e + 1023) << 52);
}
// fp64 to fp32 rounding to odd: a later rounding to e4m3 (4 significant bits)
// then gives the nearest e4m3 of the fp64 value.
__device__ __forceinline__ float to_odd(double v) {
    const float f = __double2float_rz(v);
    return ((double)f != v && isfinite(f)) ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

__device__ __forceinline__ void load8f(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// Eight channels to shared memory, asynchronously.
template <typename XT>
__device__ __forceinline__ void copy8(XT* dst, const XT* src) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(XT) / 2; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(dst) + 16 * i),
                     "l"(reinterpret_cast<const char*>(src) + 16 * i)
                     : "memory");
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {  // the low half holds a
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// cos and sin of token t's angle i, rounded to fp32: the angle in turns is
// reduced to [-1/2, 1/2] in fp64.
__device__ __forceinline__ float2 turn(int t, double turns_per_token) {
    const double x = (double)t * turns_per_token;
    float s, c;
    sincospif(2.f * (float)(x - rint(x)), &s, &c);
    return make_float2(c, s);
}
// One pair in fp64.
__device__ __noinline__ double2 exact_pair(float x, float y, int t, double freq) {
    double s, c;
    sincos((double)t * freq, &s, &c);
    return make_double2((double)x * c - (double)y * s, (double)x * s + (double)y * c);
}

// x c + y s for c = ch + cl and s = sh + sl to 2^-48, rounded to fp32 once but for
// that: products and their sum with what their roundings leave out.
__device__ __forceinline__ float rotated_once(float x, float ch, float cl, float y, float sh, float sl) {
    const float p = __fmul_rn(x, ch), q = __fmul_rn(y, sh), v = __fadd_rn(p, q);
    if (!isfinite(v)) return v;
    const float b = __fsub_rn(v, p), rest = __fadd_rn(__fsub_rn(p, __fsub_rn(v, b)), __fsub_rn(q, b));
    const float low = __fadd_rn(fmaf(x, ch, -p), fmaf(y, sh, -q));
    return __fadd_rn(v, __fadd_rn(rest, __fadd_rn(low, fmaf(x, cl, __fmul_rn(y, sl)))));
}

// The last sequence b with key(b) <= x (the first, if none has), for a key that
// grows with b: a search of 32 sequences at a time. Every lane of the warp calls
// it together.
template <typename Key>
__device__ __forceinline__ int last_at_most(int B, int64_t x, Key key) {
    const int lane = lane_id();
    int lo = 0;
    for (int n = B; n > 1;) {  // it is in [lo, lo + n)
        const int step = (n + 31) / 32, at = lane * step;
        const int k = 31 - __clz(__ballot_sync(kFull, lane == 0 || (at < n && key(lo + at) <= x)));
        lo += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    return lo;
}

// Page slot of a block: n rows touch at most n / page + 2 pages, so that the
// blocks of sequence b begin at cu_rows[b] / page + 2 b, found without a walk
// over the sequences before it (with a walk 8192 sequences of 4 rows, pages of
// 64, took 13.2 ms, now 1.4; 1024 of them 349 and 179 us; 8 x 4096 rows the same).
// False for a block that is left over, and for one of a sequence that is left
// out (seq.len < seq.rows), whose slots are its rows page by page from `slot` 0 on.
__device__ __forceinline__ bool find_item(const PagedSeqs& s, int page, int64_t item, int& b, int& slot,
                                          PagedSeq& seq) {
    auto begin = [&](int i) {
        const int64_t row = s.cu_rows ? s.cu_rows[i] : i;
        return (row < 0 ? 0 : row > s.n_rows ? s.n_rows : row) / page + 2 * (int64_t)i;
    };
    b = last_at_most(s.B, item, begin);
    seq = paged_seq(s, b);
    slot = (int)(item - begin(b));
    if (seq.rows == 0 || seq.len < seq.rows) return false;
    const int first = (seq.len - seq.rows) / page, n = (seq.len - 1) / page - first + 1;
    const int64_t at = item - begin(b);
    slot = first + (int)at;
    return at >= 0 && at < n;
}

// Zeros for query head h of packed rows [r0, r1), a warp's eight bytes a lane.
template <typename XT>
__device__ __forceinline__ void clear_rows(const PagedAppendArgs& a, int64_t r0, int64_t r1, int h) {
    constexpr int kBytes = kD * sizeof(XT);
    for (int64_t r = r0; r < r1; ++r) {
        char* at = reinterpret_cast<char*>(a.q_out) + (r * a.Hq + h) * kBytes;
        for (int i = 8 * lane_id(); i < kBytes; i += 256) *reinterpret_cast<uint2*>(at + i) = make_uint2(0, 0);
    }
}

// The codes of an older row under a grown scale: old codes are worth `ratio` new ones.
__device__ __forceinline__ void renew_row(uint8_t* at, double ratio) {
    const uint2 u = *reinterpret_cast<const uint2*>(at);
    const uint32_t w[2] = {u.x, u.y};
    uint32_t n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t f0 = e4m3x2_to_f16x2(w[i] & 0xffffu), f1 = e4m3x2_to_f16x2(w[i] >> 16);
        n[i] = e4m3x2(to_odd(f16_lo(f0) * ratio), to_odd(f16_hi(f0) * ratio)) |
               (e4m3x2(to_odd(f16_lo(f1) * ratio), to_odd(f16_hi(f1) * ratio)) << 16);
        // NaN codes are kept as they are, sign and all
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (((w[i] >> (8 * k)) & 0x7fu) == 0x7fu) n[i] = (n[i] & ~(0xffu << (8 * k))) | (w[i] & (0xffu << (8 * k)));
    }
    *reinterpret_cast<uint2*>(at) = make_uint2(n[0], n[1]);
}

// Block: one page slot (blockIdx.x / groups) and up to `a.heads` heads of K, V
// or Q (in that order of groups).
template <typename XT, int PAGE>
__global__ void __launch_bounds__(AppShape<PAGE>::kThreads)
    paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
    constexpr int kThreads = AppShape<PAGE>::kThreads, kPasses = AppShape<PAGE>::kPasses, kWarps = kThreads / 32;
    constexpr int kAhead = app_ahead<XT>();
    extern __shared__ __align__(16) float2 cs[];  // [PAGE][64] (cos, sin) of the page's rows, then the heads' rows
    __shared__ float top_sh[2][kWarps];
    __shared__ double top_exact[kWarps];
    const int l = threadIdx.x & 7, rg = threadIdx.x >> 3, lane = lane_id(), warp = threadIdx.x >> 5;
    const int gkv = (a.Hkv + a.heads - 1) / a.heads, gq = a.q ? (a.Hq + a.heads - 1) / a.heads : 0;
    const int64_t item = blockIdx.x / (2 * gkv + gq);
    int group = (int)(blockIdx.x % (2 * gkv + gq));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && a.seqs.status)
        for (int b = threadIdx.x; b < a.seqs.B; b += kThreads) paged_report(a.seqs, paged_seq(a.seqs, b).bad);
    int b = 0, slot = 0;
    PagedSeq seq{};
    const bool live = find_item(a.seqs, PAGE, item, b, slot, seq);
    const int kind = group < gkv ? 0 : group < 2 * gkv ? 1 : 2;  // K, V, Q
    const int h0 = (group - kind * gkv) * a.heads, H = kind == 2 ? a.Hq : a.Hkv;
    const int h1 = h0 + a.heads < H ? h0 + a.heads : H;
    if (!live) {
        if (kind == 2 && seq.len < seq.rows && slot >= 0 && (int64_t)slot * PAGE < seq.rows) {
            const int n = seq.rows - slot * PAGE < PAGE ? seq.rows - slot * PAGE : PAGE;
            for (int h = h0 + warp; h < h1; h += kWarps)
                clear_rows<XT>(a, (int64_t)seq.row0 + slot * PAGE, (int64_t)seq.row0 + slot * PAGE + n, h);
        }
        return;
    }
    const int start = seq.len - seq.rows, t0 = slot * PAGE;
    const int first = start > t0 ? start - t0 : 0;  // page row of the first new token
    const int last = seq.len - t0 < PAGE ? seq.len - t0 : PAGE;
    int64_t id = 0;
    if (kind < 2) {
        id = a.seqs.table[b * a.seqs.table_stride + slot];
        if (id < 0 || id >= a.num_pages) {
            if (threadIdx.x == 0) paged_report(a.seqs, kBadPage);
            return;
        }
    }
    const bool rope = a.rope && kind != 1;
    const int64_t st = kind == 0 ? a.k_st : kind == 1 ? a.v_st : a.q_st;
    const int64_t sh = kind == 0 ? a.k_sh : kind == 1 ? a.v_sh : a.q_sh;
    const XT* x0 = reinterpret_cast<const XT*>(kind == 0 ? a.k : kind == 1 ? a.v : a.q);
    const int64_t row0 = seq.row0 + t0 - start;  // packed row of page row 0
    if (sizeof(XT) == 4 && kind == 2 && rope) {
        // fp32 queries keep their 24 bits: a thread holds the angles of a row's
        // channels in two words each and takes the row's heads one after the other.
#pragma unroll 1
        for (int r = rg; r < last; r += kThreads / 8) {
            if (r < first) continue;
            float ch[8], cl[8], sh_[8], sl[8];
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
                double s, c;
                sincospi(2.0 * (t0 + r) * a.turns[8 * l + i], &s, &c);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k == i) {
                        ch[k] = (float)c, cl[k] = (float)(c - (double)ch[k]);
                        sh_[k] = (float)s, sl[k] = (float)(s - (double)sh_[k]);
                    }
            }
#pragma unroll 2
            for (int h = h0; h < h1; ++h) {
                const XT* from = x0 + h * sh + (row0 + r) * st + 8 * l;
                float x[8], y[8];
                load8f(from, x);
                load8f(from + kD / 2, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = rotated_once(x[i], ch[i], cl[i], y[i], -sh_[i], -sl[i]);
                    y[i] = rotated_once(x[i], sh_[i], sl[i], y[i], ch[i], cl[i]);
                    x[i] = u;
                }
                XT* o = reinterpret_cast<XT*>(a.q_out) + ((row0 + r) * a.Hq + h) * kD + 8 * l;
                store8(o, x);
                store8(o + kD / 2, y);
            }
        }
        return;
    }
    // The rows of the next heads are on their way to shared memory; a thread
    // reads only what it copied itself.
    XT* ring = reinterpret_cast<XT*>(cs + (a.rope ? PAGE * 64 : 0));
    auto fetch = [&](int h) {
        if (h < h1) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const int r = rg + p * (kThreads / 8);
                if (r < first || r >= last) continue;
                const XT* row = x0 + h * sh + (row0 + r) * st + 8 * l;
                XT* to = ring + (((h - h0) % kAhead) * PAGE + r) * kD + 8 * l;
                copy8(to, row);
                copy8(to + kD / 2, row + kD / 2);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) fetch(h0 + i);
    if (rope) {
        for (int i = threadIdx.x; i < (last - first) * 64; i += kThreads)
            cs[(first + (i >> 6)) * 64 + (i & 63)] = turn(t0 + first + (i >> 6), a.turns[i & 63]);
        __syncthreads();
    }
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        const XT* x = x0 + h * sh;
        float lo[kPasses][8], hi[kPasses][8];
        float top = 0.f;
        // (q_out may be q: a head's rows are all read before one of them is written)
        fetch(h + kAhead - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int r = rg + p * (kThreads / 8);
            if (r >= first && r < last) {
                const XT* from = ring + (((h - h0) % kAhead) * PAGE + r) * kD + 8 * l;
                load8f(from, lo[p]);
                load8f(from + kD / 2, hi[p]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) lo[p][i] = hi[p][i] = 0.f;
            }
        }
        if (rope) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const int r = rg + p * (kThreads / 8);
                if (r < first || r >= last) continue;
                const float4* t = reinterpret_cast<const float4*>(cs + r * 64 + 8 * l);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 w = t[i >> 1];
                    const float x0 = lo[p][i], y0 = hi[p][i], x1 = lo[p][i + 1], y1 = hi[p][i + 1];
                    lo[p][i] = fmaf(x0, w.x, -(y0 * w.y));
                    hi[p][i] = fmaf(x0, w.y, y0 * w.x);
                    lo[p][i + 1] = fmaf(x1, w.z, -(y1 * w.w));
                    hi[p][i + 1] = fmaf(x1, w.w, y1 * w.z);
                }
            }
        }
        if (kind == 2) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const int r = rg + p * (kThreads / 8);
                if (r < first || r >= last) continue;
                XT* o = reinterpret_cast<XT*>(a.q_out) + ((row0 + r) * a.Hq + h) * kD;
                store8(o + 8 * l, lo[p]);
                store8(o + kD / 2 + 8 * l, hi[p]);
            }
            continue;
        }
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // Infinities and NaN do not count; rotated in fp32, they may stand for a
                // finite value: such a page is decided in fp64 (top = infinity).
                const float u = fabsf(lo[p][i]), v = fabsf(hi[p][i]), none = rope ? INFINITY : 0.f;
                top = fmaxf(top, u < INFINITY ? u : none);
                top = fmaxf(top, v < INFINITY ? v : none);
            }
        top = warp_max(top);
        if (lane == 0) top_sh[h & 1][warp] = top;
        float* scale = (kind ? a.vs : a.ks) + id * a.Hkv + h;
        uint8_t* codes = (kind ? a.vc : a.kc) + (id * a.Hkv + h) * (int64_t)(PAGE * kD);
        const float old = first > 0 ? *scale : 0.f;
        const bool had = old > 0.f && old < INFINITY;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, top_sh[h & 1][w]);
        int e = cover_exponent(top < INFINITY ? top : 0.f);
        bool keep = had && (double)top <= 448.0 * (double)old;
        if (rope) {
            const double up = (double)top * (1.0 + (double)kErr), down = (double)top * (1.0 - (double)kErr);
            if (!(top < INFINITY) || cover_exponent(up) != cover_exponent(down) ||
                (had && (up <= 448.0 * (double)old) != (down <= 448.0 * (double)old))) {  // the whole block decides alike
                double most = 0.0;
#pragma unroll 1
                for (int r = rg; r < last; r += kThreads / 8) {
                    if (r < first) continue;
#pragma unroll 1
                    for (int i = 8 * l; i < 8 * l + 8; ++i) {
                        const XT* row = x + (row0 + r) * st;
                        const double2 v = exact_pair((float)row[i], (float)row[kD / 2 + i], t0 + r, a.freq[i]);
                        if (isfinite(v.x)) most = fmax(most, fabs(v.x));
                        if (isfinite(v.y)) most = fmax(most, fabs(v.y));
                    }
                }
#pragma unroll
                for (int m = 16; m; m >>= 1) most = fmax(most, __shfl_xor_sync(kFull, most, m));
                if (lane == 0) top_exact[warp] = most;
                __syncthreads();
                for (int w = 0; w < kWarps; ++w) most = fmax(most, top_exact[w]);
                __syncthreads();
                e = cover_exponent(most);
                keep = had && most <= 448.0 * (double)old;
            }
        }
        const double s_new = keep ? (double)old : exp2i(e);
        if (threadIdx.x == 0) *scale = (float)s_new;
        const double ratio = keep || !had ? 1.0 : (double)old / s_new;
        const double inv_d = 1.0 / s_new;
        const float inv = (float)inv_d;
        const float tiny = 0x1p-148f * inv;  // what rounding among fp32's subnormal values adds
        // a scale that is no power of two (a caller's own) has a rounded inverse
        const bool unsure = rope || (double)inv != inv_d || (__float_as_uint((float)s_new) & 0x7fffffu) != 0;
        // and a subnormal one (a caller's own) none that fp32 can hold: every code is divided in fp64
        const uint32_t all = s_new < 0x1p-126 ? 0xffffu : 0u;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int r = rg + p * (kThreads / 8);
            if (r >= last) continue;
            uint8_t* dst = codes + r * kD + 8 * l;
            if (r < first) {
                if (ratio != 1.0) {
                    renew_row(dst, ratio);
                    renew_row(dst + kD / 2, ratio);
                }
                continue;
            }
            uint32_t w[4] = {0, 0, 0, 0}, odd = all;  // odd: channels (16 of them) whose code is not sure
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float u0 = lo[p][i] * inv, u1 = lo[p][i + 1] * inv, v0 = hi[p][i] * inv, v1 = hi[p][i + 1] * inv;
                uint32_t cu, cv;
                if (unsure) {
                    const float d0 = fmaf(fabsf(u0) + fabsf(v0), kErr, tiny), d1 = fmaf(fabsf(u1) + fabsf(v1), kErr, tiny);
                    cu = e4m3x2(u0 - d0, u1 - d1);
                    cv = e4m3x2(v0 - d0, v1 - d1);
                    const uint32_t xu = cu ^ e4m3x2(u0 + d0, u1 + d1), xv = cv ^ e4m3x2(v0 + d0, v1 + d1);
                    odd |= ((xu & 0xffu ? 1u : 0u) | (xu >> 8 ? 2u : 0u) | (xv & 0xffu ? 256u : 0u) | (xv >> 8 ? 512u : 0u)) << i;
                } else {
                    cu = e4m3x2(u0, u1);
                    cv = e4m3x2(v0, v1);
                }
                w[i >> 2] |= cu << ((i & 2) * 8);
                w[2 + (i >> 2)] |= cv << ((i & 2) * 8);
            }
#pragma unroll 1
            for (; odd; odd &= odd - 1) {
                const int k = __ffs(odd) - 1, i = 8 * l + (k & 7);
                const XT* row = x + (row0 + r) * st;
                const float xa = (float)row[i], xb = (float)row[kD / 2 + i];
                double2 v = make_double2(xa, xb);
                if (rope) v = exact_pair(xa, xb, t0 + r, a.freq[i]);
                const uint32_t c = e4m3x2(to_odd((k < 8 ? v.x : v.y) / s_new), 0.f) & 0xffu;
                const int at = (k & 3) * 8;
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (m == (k >> 3) * 2 + ((k & 7) >> 2)) w[m] = (w[m] & ~(0xffu << at)) | (c << at);
            }
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(dst + kD / 2) = make_uint2(w[2], w[3]);
        }
    }
}

// The sequence of packed row r. Every lane of the warp calls it together.
__device__ __forceinline__ bool find_row(const PagedSeqs& s, int r, int& b, PagedSeq& seq) {
    b = s.cu_rows ? last_at_most(s.B, r, [&](int i) { return (int64_t)s.cu_rows[i]; }) : r;
    seq = paged_seq(s, b);
    return r >= seq.row0 && r < seq.row0 + seq.rows && seq.len >= seq.rows;
}

// The same for calls of a row or two per sequence (a decode step): a warp per
// (row, head) takes the row's page if it is the sequence's first row there, four
// rows at a time, in fp64 throughout, nothing shared. A warp finds its sequence
// in log32(B) steps: with a walk over the sequences 8192 of them took 8860 us a
// call (one row, 32 + 8 + 8 heads, pages of 64), now 470; 64 take the same.
template <typename XT>
__global__ void __launch_bounds__(128) paged_append_few_kernel(const __grid_constant__ PagedAppendArgs a) {
    __shared__ double2 turned[4][4][64];  // (cos, sin) of a warp's four rows
    const int lane = lane_id(), l = lane & 7, rg = lane >> 3;
    const int heads = 2 * a.Hkv + (a.q ? a.Hq : 0);
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t row = w / heads;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && a.seqs.status)
        for (int b = threadIdx.x; b < a.seqs.B; b += 128) paged_report(a.seqs, paged_seq(a.seqs, b).bad);
    if (row >= a.seqs.n_rows) return;
    int b = 0;
    PagedSeq seq{};
    if (!find_row(a.seqs, (int)row, b, seq)) {
        const int h = (int)(w % heads) - 2 * a.Hkv;
        if (h >= 0 && row >= seq.row0 && row < seq.row0 + seq.rows) clear_rows<XT>(a, row, row + 1, h);  // left out
        return;
    }
    const int pos = seq.len - seq.rows + (int)row - seq.row0, slot = pos / a.page;
    if (row > seq.row0 && pos % a.page) return;  // an earlier row's page
    const int hh = (int)(w % heads), kind = hh < a.Hkv ? 0 : hh < 2 * a.Hkv ? 1 : 2;  // K, V, Q
    const int h = hh - kind * a.Hkv, start = seq.len - seq.rows, t0 = slot * a.page;
    const int first = start > t0 ? start - t0 : 0, last = seq.len - t0 < a.page ? seq.len - t0 : a.page;
    const int64_t st = kind == 0 ? a.k_st : kind == 1 ? a.v_st : a.q_st;
    const int64_t sh = kind == 0 ? a.k_sh : kind == 1 ? a.v_sh : a.q_sh;
    const int64_t row0 = seq.row0 + t0 - start;
    const XT* x = reinterpret_cast<const XT*>(kind == 0 ? a.k : kind == 1 ? a.v : a.q) + h * sh + row0 * st;
    const bool rope = a.rope && kind != 1;
    // Channels [8l, 8l + 8) of both halves of this lane's row of rows r0 .. r0 + 3,
    // rotated. The whole warp computes a row's 64 angles, two a lane.
    double lo[8], hi[8];
    auto rotated = [&](int r0) {
        const int r = r0 + rg;
        float u[8], v[8];
        if (r < last) {
            load8f(x + r * st + 8 * l, u);
            load8f(x + r * st + kD / 2 + 8 * l, v);
        }
        if (rope) {
            double2(*cs)[64] = turned[threadIdx.x >> 5];
            __syncwarp();
#pragma unroll 1
            for (int k = 0; k < 4 && r0 + k < last; ++k)
#pragma unroll
                for (int i = lane; i < 64; i += 32) sincospi(2.0 * (t0 + r0 + k) * a.turns[i], &cs[k][i].y, &cs[k][i].x);
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = hi[i] = 0.0;
            if (r >= last) continue;
            lo[i] = u[i];
            hi[i] = v[i];
            if (!rope) continue;
            const double2 w = turned[threadIdx.x >> 5][rg][8 * l + i];
            lo[i] = (double)u[i] * w.x - (double)v[i] * w.y;
            hi[i] = (double)u[i] * w.y + (double)v[i] * w.x;
        }
    };
    if (kind == 2) {
#pragma unroll 1
        for (int r0 = first; r0 < last; r0 += 4) {
            const int r = r0 + rg;
            rotated(r0);
            if (r >= last) continue;
            XT* o = reinterpret_cast<XT*>(a.q_out) + ((row0 + r) * a.Hq + h) * kD + 8 * l;
            float u[8], v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // (to odd: the only rounding is the store's)
                u[i] = sizeof(XT) == 2 ? to_odd(lo[i]) : (float)lo[i];
                v[i] = sizeof(XT) == 2 ? to_odd(hi[i]) : (float)hi[i];
            }
            store8(o, u);
            store8(o + kD / 2, v);
        }
        return;
    }
    const int64_t id = a.seqs.table[b * a.seqs.table_stride + slot];
    if (id < 0 || id >= a.num_pages) {
        if (lane == 0) paged_report(a.seqs, kBadPage);
        return;
    }
    float* scale = (kind ? a.vs : a.ks) + id * a.Hkv + h;
    uint8_t* codes = (kind ? a.vc : a.kc) + (id * a.Hkv + h) * (int64_t)(a.page * kD) + 8 * l;
    const float old = first > 0 ? *scale : 0.f;
    const bool had = old > 0.f && old < INFINITY;
    double top = 0.0;
#pragma unroll 1
    for (int r0 = first; r0 < last; r0 += 4) {
        rotated(r0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (isfinite(lo[i])) top = fmax(top, fabs(lo[i]));
            if (isfinite(hi[i])) top = fmax(top, fabs(hi[i]));
        }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, m));
    const bool keep = had && top <= 448.0 * (double)old;
    const double s_new = keep ? (double)old : exp2i(cover_exponent(top));
    // a power of two is multiplied by its inverse; a caller's own scale divides
    const double inv = (__float_as_uint((float)s_new) & 0x7fffffu) ? 0.0 : 1.0 / s_new;
    auto code = [&](double a, double b) {
        return inv != 0.0 ? e4m3x2(to_odd(a * inv), to_odd(b * inv)) : e4m3x2(to_odd(a / s_new), to_odd(b / s_new));
    };
    __syncwarp();  // every lane has the old scale
    if (lane == 0) *scale = (float)s_new;
    if (!keep && had) {
        const double ratio = (double)old / s_new;
#pragma unroll 1
        for (int r = rg; r < first; r += 4) {
            renew_row(codes + r * kD, ratio);
            renew_row(codes + r * kD + kD / 2, ratio);
        }
    }
#pragma unroll 1
    for (int r0 = first; r0 < last; r0 += 4) {
        const int r = r0 + rg;
        if (last - first > 4) rotated(r0);  // else the lane still holds its one row
        if (r >= last) continue;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[i] = code(lo[4 * i], lo[4 * i + 1]) | (code(lo[4 * i + 2], lo[4 * i + 3]) << 16);
            c[2 + i] = code(hi[4 * i], hi[4 * i + 1]) | (code(hi[4 * i + 2], hi[4 * i + 3]) << 16);
        }
        *reinterpret_cast<uint2*>(codes + r * kD) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(codes + r * kD + kD / 2) = make_uint2(c[2], c[3]);
    }
}

template <typename XT>
cudaError_t launch_few(const PagedAppendArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};
    const int64_t warps = a.seqs.n_rows * (2 * a.Hkv + (a.q ? a.Hq : 0)), grid = (warps + 3) / 4;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_smem_pdl(paged_append_few_kernel<XT>, ready, dim3((unsigned)grid), dim3(128), 0, s, a);
}

template <typename XT, int PAGE>
cudaError_t launch_page(const PagedAppendArgs& a, int64_t grid, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};
    constexpr size_t ring = app_ahead<XT>() * PAGE * kD * sizeof(XT), turns = PAGE * 64 * sizeof(float2);
    return launch_smem_pdl(paged_append_kernel<XT, PAGE>, ready, dim3((unsigned)grid), dim3(AppShape<PAGE>::kThreads),
                           Smem(ring + (a.rope ? turns : 0), ring + turns), s, a);
}
template <typename XT>
cudaError_t launch_type(const PagedAppendArgs& a, int64_t grid, cudaStream_t s) {
    switch (a.page) {
        case 16: return launch_page<XT, 16>(a, grid, s);
        case 32: return launch_page<XT, 32>(a, grid, s);
        case 64: return launch_page<XT, 64>(a, grid, s);
        default: return launch_page<XT, 128>(a, grid, s);
    }
}

}  // namespace

cudaError_t launch_paged_append(PagedAppendArgs a, bool bf16, cudaStream_t s) {
    // A row or two per sequence: a page block would hold 64 threads and more to
    // each row it has (64 sequences of one row, 80 heads, pages of 64: 26 us as
    // page blocks, 12 us as a warp per page and head, both from a cold cache).
    if (a.seqs.n_rows <= 2 * (int64_t)a.seqs.B) return bf16 ? launch_few<__nv_bfloat16>(a, s) : launch_few<float>(a, s);
    // Heads per block: more of them share a page's cos and sin (computing those
    // costs a block as much as two or three heads), as long as there are four
    // blocks to an SM. Measured with two, four and eight to an SM: 5 sequences x
    // ~580 rows, fp32 33, 21, 22 us; 2 x 1000 rows 26, 26, 33 us; one of 4096
    // rows, pages of 128, 67, 61, 73 us.
    int64_t grid = 0;
    for (a.heads = 32;; a.heads /= 2) {
        const int64_t kv = (a.Hkv + a.heads - 1) / a.heads, q = a.q ? (a.Hq + a.heads - 1) / a.heads : 0;
        grid = a.items * (2 * kv + q);
        if (a.heads == 1 || grid >= 4 * (int64_t)device_sm_count()) break;
    }
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return bf16 ? launch_type<__nv_bfloat16>(a, grid, s) : launch_type<float>(a, grid, s);
}

}  // namespace nsnq
