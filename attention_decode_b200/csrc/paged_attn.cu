// Attention over the paged 8-bit cache.
//
// One block per (row, query head): its four warps take the visible tokens in
// turn, lane l holding channels [4l, 4l+4), with a running maximum and sum
// per warp that are joined at the end.
#include <math.h>

#include "attn_split.cuh"
#include "paged.cuh"

namespace nsnq {

namespace {

constexpr int kAttnThreads = 128;

template <typename QT, typename OT>
__global__ void __launch_bounds__(kAttnThreads) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
    __shared__ float sm[4], sl[4], so[4][kD];
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x / a.Hq;
    const int hq = (int)(blockIdx.x % a.Hq), h = hq / (a.Hq / a.Hkv);
    PagedSeq s{};
    int b = 0;
    bool mine = false;
    for (b = 0; b < a.seqs.B; ++b) {
        s = paged_seq(a.seqs, b);
        if (blockIdx.x == 0 && threadIdx.x == 0)
            paged_report(a.seqs, s.bad | (s.rows > a.max_rows ? kBadLength : 0u));
        if (r >= s.row0 && r < s.row0 + s.rows && r - s.row0 < a.max_rows) mine = true;
        if (mine && blockIdx.x) break;
    }
    if (blockIdx.x == 0)
        for (b = 0; b < a.seqs.B; ++b) {
            s = paged_seq(a.seqs, b);
            if (r >= s.row0 && r < s.row0 + s.rows && r - s.row0 < a.max_rows) break;
        }
    if (!mine) return;
    const int pos = s.len - s.rows + (int)(r - s.row0);
    float q[4];
    load4(reinterpret_cast<const QT*>(a.q) + r * a.q_st + hq * a.q_sh + 4 * lane, q);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
    const int ns = a.sinks < lo ? a.sinks : lo;  // sinks in front of the window
    for (int i = warp; i < ns + pos + 1 - lo; i += 4) {
        const int t = i < ns ? i : i - ns + lo;
        const int64_t id = a.seqs.table[b * a.seqs.table_stride + t / a.page];
        if (id < 0 || id >= a.num_pages) {
            if (lane == 0) paged_report(a.seqs, kBadPage);
            continue;
        }
        const int64_t ph = id * a.Hkv + h;
        const int64_t at = (ph * a.page + t % a.page) * kD + 4 * lane;
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(a.kc + at);
        const uint32_t vw = *reinterpret_cast<const uint32_t*>(a.vc + at);
        const uint32_t k0 = e4m3x2_to_f16x2(kw & 0xffffu), k1 = e4m3x2_to_f16x2(kw >> 16);
        float dot = q[0] * f16_lo(k0);
        dot = fmaf(q[1], f16_hi(k0), dot);
        dot = fmaf(q[2], f16_lo(k1), dot);
        dot = fmaf(q[3], f16_hi(k1), dot);
        const float sc = warp_sum(dot) * (a.ks[ph] * a.scale_log2);
        const float mn = fmaxf(m, sc);
        const float f = m == mn ? 1.f : exp2f(m - mn), p = exp2f(sc - mn);
        m = mn;
        l = fmaf(l, f, p);
        const float w = p * a.vs[ph];
        const uint32_t v0 = e4m3x2_to_f16x2(vw & 0xffffu), v1 = e4m3x2_to_f16x2(vw >> 16);
        const float v[4] = {f16_lo(v0), f16_hi(v0), f16_lo(v1), f16_hi(v1)};
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = fmaf(w, v[k], o[k] * f);
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int k = 0; k < 4; ++k) so[warp][4 * lane + k] = o[k];
    __syncthreads();
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float total = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = sl[w] == 0.f ? 0.f : exp2f(sm[w] - top);
        total += f * sl[w];
        acc += sl[w] == 0.f ? 0.f : f * so[w][threadIdx.x];
    }
    const float y = total == 0.f ? 0.f : acc / total;
    const int64_t at = (r * a.Hq + hq) * kD + threadIdx.x;
    if constexpr (sizeof(OT) == 2) reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
    else reinterpret_cast<float*>(a.out)[at] = y;
}

}  // namespace

size_t paged_attn_workspace(int64_t, int, int, int, int64_t) { return 256; }

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.seqs.n_rows * a.Hq);
    if (a.q_bf16) {
        if (a.out_bf16) paged_attn_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kAttnThreads, 0, s>>>(a);
        else paged_attn_kernel<__nv_bfloat16, float><<<grid, kAttnThreads, 0, s>>>(a);
    } else {
        if (a.out_bf16) paged_attn_kernel<float, __nv_bfloat16><<<grid, kAttnThreads, 0, s>>>(a);
        else paged_attn_kernel<float, float><<<grid, kAttnThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace nsnq
