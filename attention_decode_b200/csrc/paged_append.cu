// Append to the paged 8-bit cache: new keys and values, the keys (and
// queries) rotated to their positions, stored in e4m3 under one power-of-two
// scale per (page, head).
//
// x -> code = e4m3(x / 2^e), e the least exponent with every |x| of the
// (page, head) <= 448 * 2^e. One block owns one (page, head) of K or V, so
// the page's scale, the codes of its new tokens and, where the scale grows,
// the renewed codes of its older tokens have a single writer and no atomics.
#include <math.h>

#include "paged.cuh"

namespace nsnq {

namespace {

constexpr int kAppThreads = 128;  // 16 rows of 8 lanes; a lane holds channels [8l, 8l+8) of both halves

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

template <typename XT>
__device__ __forceinline__ void load8f(const XT* p, float (&v)[8]) {
    float a[4], b[4];
    load4(p, a);
    load4(p + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void store8(float* p, const double (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = (float)v[i];
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const double (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = (uint32_t)f32_to_bf16_rn(to_odd(v[2 * i])) | ((uint32_t)f32_to_bf16_rn(to_odd(v[2 * i + 1])) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Channels [8l, 8l+8) and [64+8l, 64+8l+8) of one row, rotated to position t.
template <typename XT>
__device__ __forceinline__ void load_rotated(const PagedAppendArgs& a, const XT* row, int l, int t, bool rope,
                                             double (&lo)[8], double (&hi)[8]) {
    float x[8], y[8];
    load8f(row + 8 * l, x);
    load8f(row + kD / 2 + 8 * l, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = x[i];
        hi[i] = y[i];
        if (rope) {
            double s, c;
            sincos((double)t * a.freq[8 * l + i], &s, &c);
            lo[i] = (double)x[i] * c - (double)y[i] * s;
            hi[i] = (double)x[i] * s + (double)y[i] * c;
        }
    }
}

__device__ __forceinline__ double block_max(double v, double* sh) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, m));
    if (lane_id() == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = fmax(fmax(sh[0], sh[1]), fmax(sh[2], sh[3]));
    return v;
}

// The item'th page slot that the call writes: sequences in order, each with
// the slots its new rows touch. Every thread of a warp calls it together.
__device__ __forceinline__ bool find_item(const PagedSeqs& s, int page, int64_t item, int& b, int& slot,
                                          PagedSeq& seq) {
    const int lane = lane_id();
    int64_t before = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
        PagedSeq q{};
        int n = 0, first = 0;
        if (b0 + lane < s.B) {
            q = paged_seq(s, b0 + lane);
            if (q.rows > 0 && q.len >= q.rows) {
                first = (q.len - q.rows) / page;
                n = (q.len - 1) / page - first + 1;
            }
        }
        int64_t incl = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(kFull, incl, m);
            if (lane >= m) incl += o;
        }
        const unsigned hit = __ballot_sync(kFull, item < before + incl);
        if (hit) {
            const int src = __ffs(hit) - 1;
            b = b0 + src;
            const int64_t lead = __shfl_sync(kFull, incl - n, src);
            slot = (int)(item - before - lead) + __shfl_sync(kFull, first, src);
            seq.row0 = __shfl_sync(kFull, q.row0, src);
            seq.rows = __shfl_sync(kFull, q.rows, src);
            seq.len = __shfl_sync(kFull, q.len, src);
            return true;
        }
        before += __shfl_sync(kFull, incl, 31);
    }
    return false;
}

template <typename XT>
__global__ void __launch_bounds__(kAppThreads) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
    __shared__ double sh[4];
    const int l = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const int64_t page_blocks = a.items * 2 * a.Hkv;
    if (blockIdx.x >= page_blocks) {  // queries: 16 rows of one head
        const int64_t qb = blockIdx.x - page_blocks;
        const int64_t r = qb / a.Hq * 16 + rg;
        const int h = (int)(qb % a.Hq);
        if (r >= a.seqs.n_rows) return;
        int t = 0;
        bool mine = false;
        for (int b = 0; b < a.seqs.B && !mine; ++b) {
            const PagedSeq s = paged_seq(a.seqs, b);
            mine = r >= s.row0 && r < s.row0 + s.rows && s.len >= s.rows;
            t = s.len - s.rows + (int)(r - s.row0);
        }
        if (!mine) return;
        double lo[8], hi[8];
        load_rotated(a, reinterpret_cast<const XT*>(a.q) + r * a.q_st + h * a.q_sh, l, t, a.rope != 0, lo, hi);
        XT* o = reinterpret_cast<XT*>(a.q_out) + (r * a.Hq + h) * kD;
        store8(o + 8 * l, lo);
        store8(o + kD / 2 + 8 * l, hi);
        return;
    }
    const int64_t item = blockIdx.x / (2 * a.Hkv);
    const int hh = (int)(blockIdx.x % (2 * a.Hkv));
    if (blockIdx.x == 0 && a.seqs.status)
        for (int b = threadIdx.x; b < a.seqs.B; b += kAppThreads) paged_report(a.seqs, paged_seq(a.seqs, b).bad);
    const bool is_v = hh >= a.Hkv;
    const int h = is_v ? hh - a.Hkv : hh;
    int b = 0, slot = 0;
    PagedSeq seq{};
    if (!find_item(a.seqs, a.page, item, b, slot, seq)) return;
    const int64_t id = a.seqs.table[b * a.seqs.table_stride + slot];
    if (id < 0 || id >= a.num_pages) {
        if (threadIdx.x == 0 && hh == 0) paged_report(a.seqs, kBadPage);
        return;
    }
    const int start = seq.len - seq.rows;
    const int first = start > slot * a.page ? start - slot * a.page : 0;  // page row of the first new token
    const int last = seq.len - slot * a.page < a.page ? seq.len - slot * a.page : a.page;
    const XT* x = is_v ? reinterpret_cast<const XT*>(a.v) + h * a.v_sh : reinterpret_cast<const XT*>(a.k) + h * a.k_sh;
    const int64_t st = is_v ? a.v_st : a.k_st;
    const bool rope = a.rope && !is_v;
    double top = 0.0;
    double lo[8], hi[8];
    for (int r = rg; r < a.page; r += 16) {
        if (r < first || r >= last) continue;
        const int t = slot * a.page + r;
        load_rotated(a, x + (int64_t)(seq.row0 + t - start) * st, l, t, rope, lo, hi);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (isfinite(lo[i])) top = fmax(top, fabs(lo[i]));
            if (isfinite(hi[i])) top = fmax(top, fabs(hi[i]));
        }
    }
    top = block_max(top, sh);
    float* scale = (is_v ? a.vs : a.ks) + id * a.Hkv + h;
    uint8_t* codes = (is_v ? a.vc : a.kc) + (id * a.Hkv + h) * (int64_t)a.page * kD;
    double s_new = exp2i(cover_exponent(top));
    double ratio = 1.0;  // old codes are worth ratio new ones
    if (first > 0) {
        const float old = *scale;
        if (old > 0.f && isfinite(old)) {
            if (top <= 448.0 * (double)old) s_new = (double)old;
            else ratio = (double)old / s_new;
        }
    }
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *scale = (float)s_new;
    const double inv = 1.0 / s_new;
    for (int r = rg; r < last; r += 16) {
        uint8_t* dst = codes + r * kD;
        if (r < first) {
            if (ratio == 1.0) continue;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint2 u = *reinterpret_cast<const uint2*>(dst + p * (kD / 2) + 8 * l);
                uint32_t w[2] = {u.x, u.y}, n[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t f0 = e4m3x2_to_f16x2(w[i] & 0xffffu), f1 = e4m3x2_to_f16x2(w[i] >> 16);
                    n[i] = e4m3x2(to_odd(f16_lo(f0) * ratio), to_odd(f16_hi(f0) * ratio)) |
                           (e4m3x2(to_odd(f16_lo(f1) * ratio), to_odd(f16_hi(f1) * ratio)) << 16);
                }
                *reinterpret_cast<uint2*>(dst + p * (kD / 2) + 8 * l) = make_uint2(n[0], n[1]);
            }
            continue;
        }
        const int t = slot * a.page + r;
        load_rotated(a, x + (int64_t)(seq.row0 + t - start) * st, l, t, rope, lo, hi);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[i] = e4m3x2(to_odd(lo[4 * i] * inv), to_odd(lo[4 * i + 1] * inv)) |
                   (e4m3x2(to_odd(lo[4 * i + 2] * inv), to_odd(lo[4 * i + 3] * inv)) << 16);
            w[2 + i] = e4m3x2(to_odd(hi[4 * i] * inv), to_odd(hi[4 * i + 1] * inv)) |
                       (e4m3x2(to_odd(hi[4 * i + 2] * inv), to_odd(hi[4 * i + 3] * inv)) << 16);
        }
        *reinterpret_cast<uint2*>(dst + 8 * l) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + kD / 2 + 8 * l) = make_uint2(w[2], w[3]);
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, bool bf16, cudaStream_t s) {
    const int64_t qblocks = a.q ? (a.seqs.n_rows + 15) / 16 * a.Hq : 0;
    const int64_t grid = a.items * 2 * a.Hkv + qblocks;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (bf16) paged_append_kernel<__nv_bfloat16><<<(unsigned)grid, kAppThreads, 0, s>>>(a);
    else paged_append_kernel<float><<<(unsigned)grid, kAppThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace nsnq
