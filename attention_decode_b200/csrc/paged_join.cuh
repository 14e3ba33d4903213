// Shared by the two paged attention kernels: their arguments, the parts that
// a CTA leaves in the workspace for a unit it did not finish, and the kernel
// that joins them.
#pragma once

#include "attn_split.cuh"
#include "paged_plan.cuh"
#include "umma.cuh"

namespace nsnq {

// Prompt rows: paged_rows.cu.
cudaError_t launch_paged_rows(const PagedAttnArgs& a, cudaStream_t s);
size_t paged_rows_workspace();

// A part of a unit of RC rows: [RC][128] outputs over the part's tokens alone (of
// the values' own size, whatever the scales), [RC] m, [RC] l, the sum of the
// weights relative to 2^m. A CTA leaves at most two: slot 2c for the unit its range begins in, 2c + 1 for a later one.
template <int RC>
__host__ __device__ constexpr int64_t part_stride() { return RC * (kD + 2); }

// Bytes of a workspace for `ctas` CTAs: a seam each, then two parts each.
template <int RC>
__host__ __device__ constexpr size_t paged_workspace(int ctas) {
    return (size_t)ctas * 32 + (size_t)2 * ctas * part_stride<RC>() * sizeof(float);
}
// The arguments with the workspace laid out for `ctas` CTAs.
inline PagedAttnArgs paged_lay_out(PagedAttnArgs a, int ctas) {
    a.seams = static_cast<PagedSeam*>(a.workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + (size_t)ctas * 32);
    return a;
}

struct MapPair {
    CUtensorMap k, v;
};

#ifdef __CUDACC__

static_assert(sizeof(PagedSeam) == 32, "seam layout");

__device__ __forceinline__ void store_out(const PagedAttnArgs& a, int64_t row, int d, float v) {
    if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[row * kD + d] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(a.out)[row * kD + d] = v;
}

// Waits until a limit; once a wait has failed, the kernel goes through the
// motions without waiting (every index is still in bounds) and the call's
// results are void: it reports that.
struct Waiter {
    bool good = true;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) {
        if (good) good = mbar_wait(bar, parity);
    }
};

constexpr int kJoinThreads = 128;
constexpr int kMaxParts = 640;  // CTAs of the largest grid (two per SM of up to 320) and one more

// Block (c, y), c < grid: where a unit crosses into CTA c and began in c - 1,
// joins rows of it, lane = 4 channels. A unit of few rows may be in many parts
// (a long context over every CTA): the four warps then share a row's parts, in
// a fixed order. A unit of many rows is in two or three: a warp takes a row.
// Block (grid + b, y): zeros for the rows of sequence b in front of its first
// token, and the report of its lengths.
template <int RC>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, int grid) {
    constexpr int kWarps = kJoinThreads / 32, kShare = RC <= 16 ? kWarps : 1;  // warps to a row
    __shared__ float factor[kWarps][kMaxParts / kShare + 1];
    __shared__ float4 sums[kWarps][32];
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x >= grid) {
        const PagedSeq s = paged_seq(a.seqs, blockIdx.x - grid);
        if (blockIdx.y == 0 && threadIdx.x == 0) paged_report(a.seqs, s.bad | (s.rows > a.max_rows ? kBadLength : 0u));
        const int64_t rows = s.rows < a.max_rows ? s.rows : a.max_rows;
        const int64_t blind = s.rows - s.len < rows ? s.rows - s.len : rows;
#pragma unroll 1
        for (int64_t i = blockIdx.y; i < blind * a.Hq; i += gridDim.y)
            store_out(a, (int64_t)s.row0 * a.Hq + i, threadIdx.x, 0.f);
        return;
    }
    const PagedSeam seam = a.seams[blockIdx.x];
    const int r = blockIdx.y * (kWarps / kShare) + warp / kShare;
    if (!seam.live || r >= seam.rows) return;  // (with shared rows, the whole block)
    const int c = blockIdx.x, n = seam.last - c + 2, w0 = warp % kShare;
    auto part = [&](int k) { return a.part + (k ? 2 * (c + k - 1) : seam.first) * part_stride<RC>(); };
    float top = -INFINITY;
    for (int k = lane; k < n; k += 32) {
        const float* p = part(k) + RC * kD + r;
        const float m = p[0], l = p[RC];
        if (l != 0.f) top = fmaxf(top, m);
    }
    top = warp_max(top);
    float sum = 0.f;
    for (int k = lane; k < n; k += 32) {
        const float* p = part(k) + RC * kD + r;
        const float m = p[0], l = p[RC];
        const float f = l != 0.f ? exp2_approx(m - top) * l : -1.f;  // -1: the row sees nothing of the part
        if (k % kShare == w0) factor[warp][k / kShare] = f;
        if (l != 0.f) sum += f;
    }
    sum = warp_sum(sum);
    __syncwarp();
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = w0; k < n; k += kShare) {
        const float4 v = *reinterpret_cast<const float4*>(part(k) + r * kD + 4 * lane);
        const float f = factor[warp][k / kShare];
        const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)  // a factor of 0 keeps the part's NaN, and nothing else of it
            if (f != -1.f && (f != 0.f || isnan(w[i]))) acc[i] = fmaf(f * inv, w[i], acc[i]);
    }
    if (kShare > 1) {
        sums[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int w = 1; w < kShare; ++w) {
            const float4 v = sums[w][lane];
            acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
        }
    }
    const int rr = seam.r0 + r, i = (int)fdiv((uint32_t)rr, a.G), G = (int)a.G.d;
    const int64_t at = ((int64_t)(seam.row0 + i) * a.Hq + seam.h * G + rr - i * G) * kD + 4 * lane;
    if (a.out_bf16)
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) =
            make_uint2((uint32_t)f32_to_bf16_rn(acc[0]) | ((uint32_t)f32_to_bf16_rn(acc[1]) << 16),
                       (uint32_t)f32_to_bf16_rn(acc[2]) | ((uint32_t)f32_to_bf16_rn(acc[3]) << 16));
    else
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(acc[0], acc[1], acc[2], acc[3]);
}

template <int RC>
cudaError_t launch_paged_join(const PagedAttnArgs& a, int grid, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};
    return launch_smem_pdl(paged_join_kernel<RC>, ready, dim3(grid + a.seqs.B, RC <= 16 ? RC : RC / 4), dim3(kJoinThreads), 0, s, a,
                           grid);
}

#endif  // __CUDACC__

}  // namespace nsnq
